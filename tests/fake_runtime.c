/* A CUDA runtime for tests without a GPU: one sm_100 device whose launches are
 * counted and never run, and whose memory is what fake_known() was told.  Loaded
 * with RTLD_GLOBAL before the library, it stands in for the real runtime's
 * functions of the same names. */
#include <stddef.h>
#include <stdint.h>
#include <string.h>

static long launches, allocs;
static uintptr_t known_lo, known_hi;
static uint64_t word[512];

void fake_known(uintptr_t lo, uintptr_t hi) { known_lo = lo, known_hi = hi; }
long fake_launches(void) { return launches; }
long fake_allocs(void) { return allocs; }

int cudaGetDevice(int* dev) { return *dev = 0, 0; }
int cudaDeviceGetAttribute(int* v, int attr, int dev) {
  (void)dev;
  *v = attr == 75 ? 10 : attr == 76 ? 0 : attr == 16 ? 148 : 0; /* capability 10.0, SMs */
  return 0;
}
int cudaGetLastError(void) { return 0; }
int cudaThreadExchangeStreamCaptureMode(int* mode) { return (void)mode, 0; }
int cudaGetSymbolAddress(void** p, const void* s) { return (void)s, *p = word, 0; }
struct attributes {
  int type, device;
  void *device_pointer, *host_pointer;
  long reserved[8];
};
int cudaPointerGetAttributes(struct attributes* a, const void* p) {
  const uintptr_t x = (uintptr_t)p;
  a->type = x >= known_lo && x < known_hi ? 2 : 0; /* device memory, or not registered */
  a->device = 0;
  a->device_pointer = a->host_pointer = NULL;
  return 0;
}
int cudaMallocAsync(void** p, size_t n, void* st) { return (void)n, (void)st, *p = (void*)(uintptr_t)0x700000000000, ++allocs, 0; }
int cudaFreeAsync(void* p, void* st) { return (void)p, (void)st, 0; }
int cudaFuncSetAttribute(const void* f, int a, int v) { return (void)f, (void)a, (void)v, 0; }
int cudaMemset(void* p, int v, size_t n) { return (void)p, (void)v, (void)n, 0; }
int cudaMemcpyAsync(void* d, const void* s, size_t n, int k, void* st) { return (void)d, (void)s, (void)n, (void)k, (void)st, ++launches, 0; }
int cudaMemcpy2DAsync(void* d, size_t dp, const void* s, size_t sp, size_t w, size_t h, int k, void* st) {
  return (void)d, (void)dp, (void)s, (void)sp, (void)w, (void)h, (void)k, (void)st, ++launches, 0;
}
int cudaStreamSynchronize(void* st) { return (void)st, 0; }
typedef struct {
  unsigned x, y, z;
} dim3_;
static dim3_ cfg_grid, cfg_block;
unsigned __cudaPushCallConfiguration(dim3_ g, dim3_ b, size_t smem, void* st) {
  return (void)smem, (void)st, cfg_grid = g, cfg_block = b, 0;
}
int __cudaPopCallConfiguration(dim3_* g, dim3_* b, size_t* smem, void** st) {
  return *g = cfg_grid, *b = cfg_block, *smem = 0, *st = NULL, 0;
}
int cudaLaunchKernel(const void* f, dim3_ g, dim3_ b, void** args, size_t smem, void* st) {
  return (void)f, (void)g, (void)b, (void)args, (void)smem, (void)st, ++launches, 0;
}
int cudaLaunchKernelExC(const void* c, const void* f, void** args) { return (void)c, (void)f, (void)args, ++launches, 0; }
