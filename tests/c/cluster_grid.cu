// The persistent cluster grid's host side with a runtime of its own: the calls that
// cluster_grid makes are defined beside this file, so that nothing needs a GPU.
#include <cstdio>

#include "umma.cuh"

// "Kernels" of one type, and the runtime's state (cluster_grid_runtime.cpp).
void wide(int);
void narrow(int);
void never(int);
extern int device, asked;

#define EXPECT(x)                                        \
    if (!(x)) {                                          \
        std::printf("line %d: %s\n", __LINE__, #x);      \
        return 1;                                        \
    }

int main()
{
    using ep::cluster_grid;
    EXPECT(cluster_grid(wide, 192, 1000, 152) == 152);
    EXPECT(cluster_grid(narrow, 192, 1000, 152) == 80);
    EXPECT(cluster_grid(never, 192, 1000, 152) == 0);
    EXPECT(cluster_grid(wide, 192, 1000, 152) == 152);
    EXPECT(cluster_grid(wide, 192, 1000, 101) == 100);
    EXPECT(cluster_grid(narrow, 192, 1000, 60) == 60);
    EXPECT(asked == 3);                                  // once per kernel that fits
    device = 1;
    EXPECT(cluster_grid(wide, 192, 1000, 152) == 150);
    device = 0;
    EXPECT(cluster_grid(wide, 192, 1000, 152) == 152);
    EXPECT(asked == 4);
    return 0;
}
