// Stands in for the HIP runtime's launches: none reaches a device, and number stub_fail_at fails.
#include <stddef.h>

extern "C" {

struct Dim {
    unsigned x, y, z;
};

static int launches, fail_at, last;

void stub_reset(int at) { launches = last = 0, fail_at = at; }
int stub_launches() { return launches; }

int __hipPushCallConfiguration(Dim, Dim, size_t, void*) { return 0; }
int __hipPopCallConfiguration(Dim* grid, Dim* block, size_t* shared, void** stream) {
    *grid = *block = Dim{1, 1, 1};
    *shared = 0;
    *stream = nullptr;
    return 0;
}
int hipLaunchKernel(const void*, Dim, Dim, void**, size_t, void*) {
    if (++launches == fail_at) last = 1;
    return last;
}
int hipGetLastError() {
    const int e = last;
    last = 0;
    return e;
}
}
