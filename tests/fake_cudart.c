/*
 * A stand-in for the CUDA runtime, for tests of the library's host side without
 * a GPU: linked with the library's objects in place of the runtime, it counts
 * devices, keeps attributes by kernel and device as the runtime does, refuses
 * launches beyond them, and writes down what was launched.  "Device memory" is
 * host memory.  No kernel runs but one of two words, which takes the products'
 * status and is carried out here by its definition.
 */
#include <cuda.h>
#include <cuda_runtime_api.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

enum { kMost = 512, kDevices = 4, kDefaultSmem = 48 * 1024 };

typedef struct {
  int device;
  unsigned grid, block, cluster;
  size_t smem;
  int overlaps; /* programmatic stream serialization */
  char name[256];
} launch_t;

static int current;
static launch_t launches[kMost];
static int num_launches;
static struct {
  const void *func;
  char name[256];
  int smem[kDevices];
} kernels[kMost];
static int num_kernels;
static struct {
  const void *symbol;
  char name[256];
  unsigned char memory[kDevices][256];
} symbols[32];
static int num_symbols;
static unsigned *late_word, late_bits;
static char fail_name[64];
static int fail_count, fail_code;

/* ---- for the test ---- */

void fake_reset(void) {
  current = num_launches = fail_count = 0;
  late_bits = 0;
  for (int i = 0; i < num_kernels; ++i)
    for (int d = 0; d < kDevices; ++d) kernels[i].smem[d] = kDefaultSmem;
}
void fake_use_device(int device) { current = device; }
/* The products' status word on the current device. */
unsigned *fake_status(void) {
  for (int i = 0; i < num_symbols; ++i)
    if (strstr(symbols[i].name, "g_ops_status")) return (unsigned *)symbols[i].memory[current];
  abort();
}
/* `bits` come into the status right after the next copy to the host. */
void fake_late(unsigned bits) { late_word = fake_status(), late_bits = bits; }
/* The next `count` calls of `name` return `code`. */
void fake_fail(const char *name, int code, int count) {
  snprintf(fail_name, sizeof fail_name, "%s", name);
  fail_code = code;
  fail_count = count;
}
int fake_launches(void) { return num_launches; }
const launch_t *fake_launch(int i) { return &launches[i]; }

static int failing(const char *name) {
  if (fail_count == 0 || strcmp(name, fail_name) != 0) return 0;
  --fail_count;
  return fail_code;
}
#define MAY_FAIL(name) \
  do { \
    int e_ = failing(name); \
    if (e_ != 0) return (cudaError_t)e_; \
  } while (0)

/* ---- registration ---- */

void **__cudaRegisterFatBinary(void *fat) {
  (void)fat;
  static void *handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void **h) { (void)h; }
void __cudaUnregisterFatBinary(void **h) { (void)h; }
void __cudaRegisterFunction(void **h, const char *host, char *device, const char *name, int limit, void *tid, void *bid,
                            void *block, void *grid, int *warp) {
  (void)h, (void)device, (void)limit, (void)tid, (void)bid, (void)block, (void)grid, (void)warp;
  if (num_kernels == kMost) abort();
  kernels[num_kernels].func = host;
  snprintf(kernels[num_kernels].name, sizeof kernels[0].name, "%s", name);
  for (int d = 0; d < kDevices; ++d) kernels[num_kernels].smem[d] = kDefaultSmem;
  ++num_kernels;
}
void __cudaRegisterVar(void **h, char *host, char *device, const char *name, int ext, size_t size, int constant,
                       int global) {
  (void)h, (void)device, (void)ext, (void)constant, (void)global;
  if (num_symbols == 32 || size > sizeof symbols[0].memory[0]) return;
  snprintf(symbols[num_symbols].name, sizeof symbols[0].name, "%s", name);
  symbols[num_symbols++].symbol = host;
}
static int kernel_of(const void *func) {
  for (int i = 0; i < num_kernels; ++i)
    if (kernels[i].func == func) return i;
  return -1;
}

/* ---- launches ---- */

static cudaError_t note(const void *func, unsigned grid, unsigned block, unsigned cluster, size_t smem, int overlaps) {
  const int k = kernel_of(func);
  if (k < 0 || num_launches == kMost) return cudaErrorInvalidDeviceFunction;
  if (smem > (size_t)kernels[k].smem[current]) return cudaErrorInvalidValue;
  launch_t *l = &launches[num_launches++];
  l->device = current, l->grid = grid, l->block = block, l->cluster = cluster, l->smem = smem, l->overlaps = overlaps;
  memcpy(l->name, kernels[k].name, sizeof l->name);
  return cudaSuccess;
}
/* Reports a timeout (8) before a capacity error (4), clears what is reported, leaves the rest. */
static void take_status(void **args) {
  struct {
    unsigned *status, *taken;
  } d;
  memcpy(&d, args[0], sizeof d);
  *d.taken = *d.status & 8 ? 8 : *d.status & 4;
  *d.status &= ~*d.taken;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *func, void **args) {
  MAY_FAIL("cudaLaunchKernelExC");
  const int k = kernel_of(func);
  if (k >= 0 && strstr(kernels[k].name, "take_status")) take_status(args);
  unsigned cluster = 1;
  int overlaps = 0;
  for (unsigned i = 0; i < c->numAttrs; ++i) {
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = c->attrs[i].val.clusterDim.x;
    if (c->attrs[i].id == cudaLaunchAttributeProgrammaticStreamSerialization)
      overlaps = c->attrs[i].val.programmaticStreamSerializationAllowed;
  }
  return note(func, c->gridDim.x, c->blockDim.x, cluster, c->dynamicSmemBytes, overlaps);
}
static struct {
  dim3 grid, block;
  size_t smem;
  cudaStream_t stream;
} pushed;
unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t smem, cudaStream_t stream) {
  pushed.grid = grid, pushed.block = block, pushed.smem = smem, pushed.stream = stream;
  return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3 *grid, dim3 *block, size_t *smem, void *stream) {
  *grid = pushed.grid, *block = pushed.block, *smem = pushed.smem, *(cudaStream_t *)stream = pushed.stream;
  return cudaSuccess;
}
cudaError_t __cudaGetKernel(cudaKernel_t *kernel, const void *func) {
  *kernel = (cudaKernel_t)func;
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t kernel, dim3 grid, dim3 block, void **args, size_t smem, cudaStream_t stream) {
  (void)args, (void)stream;
  return note(kernel, grid.x, block.x, 1, smem, 0);
}
cudaError_t cudaLaunchCooperativeKernel(const void *func, dim3 grid, dim3 block, void **args, size_t smem,
                                        cudaStream_t stream) {
  (void)args, (void)stream;
  return note(func, grid.x, block.x, 1, smem, 0);
}
cudaError_t cudaFuncSetAttribute(const void *func, enum cudaFuncAttribute attr, int value) {
  MAY_FAIL("cudaFuncSetAttribute");
  const int k = kernel_of(func);
  if (k < 0) return cudaErrorInvalidDeviceFunction;
  if (attr == cudaFuncAttributeMaxDynamicSharedMemorySize) kernels[k].smem[current] = value;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *func, const cudaLaunchConfig_t *c) {
  MAY_FAIL("cudaOccupancyMaxActiveClusters");
  const int k = kernel_of(func);
  if (k < 0 || c->dynamicSmemBytes > (size_t)kernels[k].smem[current]) return cudaErrorInvalidValue;
  *n = 60 + current; /* not the same on every device */
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int *n, const void *f, int block, size_t smem, unsigned fl) {
  (void)f, (void)block, (void)smem, (void)fl;
  *n = 1;
  return cudaSuccess;
}

/* ---- devices, memory, streams ---- */

cudaError_t cudaGetDevice(int *device) {
  MAY_FAIL("cudaGetDevice");
  *device = current;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int *v, enum cudaDeviceAttr attr, int device) {
  (void)device;
  *v = attr == cudaDevAttrMultiProcessorCount ? 152 : attr == cudaDevAttrMaxSharedMemoryPerBlockOptin ? 232448 : 0;
  return cudaSuccess;
}
static CUresult encode(CUtensorMap *map, CUtensorMapDataType type, cuuint32_t rank, void *at, const cuuint64_t *dims,
                       const cuuint64_t *strides, const cuuint32_t *box, const cuuint32_t *steps,
                       CUtensorMapInterleave i, CUtensorMapSwizzle s, CUtensorMapL2promotion p, CUtensorMapFloatOOBfill f) {
  (void)type, (void)rank, (void)at, (void)dims, (void)strides, (void)box, (void)steps, (void)i, (void)s, (void)p, (void)f;
  memset(map, 0, sizeof *map);
  return CUDA_SUCCESS;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char *name, void **f, unsigned version, unsigned long long flags,
                                             enum cudaDriverEntryPointQueryResult *r) {
  (void)name, (void)version, (void)flags;
  MAY_FAIL("cudaGetDriverEntryPointByVersion");
  *f = (void *)encode;
  *r = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void **at, const void *symbol) {
  MAY_FAIL("cudaGetSymbolAddress");
  for (int i = 0; i < num_symbols; ++i)
    if (symbols[i].symbol == symbol) {
      *at = symbols[i].memory[current];
      return cudaSuccess;
    }
  return cudaErrorInvalidSymbol;
}
cudaError_t cudaMemcpy(void *to, const void *from, size_t n, enum cudaMemcpyKind kind) {
  memcpy(to, from, n);
  if (kind == cudaMemcpyDeviceToHost && late_bits) *late_word |= late_bits, late_bits = 0;
  return cudaSuccess;
}
cudaError_t cudaMemcpyAsync(void *to, const void *from, size_t n, enum cudaMemcpyKind kind, cudaStream_t s) {
  (void)s;
  MAY_FAIL("cudaMemcpyAsync");
  return cudaMemcpy(to, from, n, kind);
}
cudaError_t cudaMemsetAsync(void *to, int v, size_t n, cudaStream_t s) {
  (void)s;
  memset(to, v, n);
  return cudaSuccess;
}
cudaError_t cudaMallocAsync(void **p, size_t n, cudaStream_t s) {
  (void)s;
  *p = calloc(1, n);
  return *p ? cudaSuccess : cudaErrorMemoryAllocation;
}
cudaError_t cudaFreeAsync(void *p, cudaStream_t s) {
  (void)s;
  free(p);
  return cudaSuccess;
}
cudaError_t cudaHostAlloc(void **p, size_t n, unsigned flags) {
  (void)flags;
  *p = calloc(1, n);
  return *p ? cudaSuccess : cudaErrorMemoryAllocation;
}
cudaError_t cudaFreeHost(void *p) {
  free(p);
  return cudaSuccess;
}
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaDeviceGetDefaultMemPool(cudaMemPool_t *pool, int device) {
  (void)device;
  *pool = NULL;
  return cudaSuccess;
}
cudaError_t cudaMemPoolSetAttribute(cudaMemPool_t pool, enum cudaMemPoolAttr attr, void *v) {
  (void)pool, (void)attr, (void)v;
  return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t s) {
  (void)s;
  MAY_FAIL("cudaStreamSynchronize");
  return cudaSuccess;
}
cudaError_t cudaStreamCreateWithFlags(cudaStream_t *s, unsigned flags) { return (void)flags, *s = NULL, cudaSuccess; }
cudaError_t cudaStreamDestroy(cudaStream_t s) { return (void)s, cudaSuccess; }
cudaError_t cudaStreamWaitEvent(cudaStream_t s, cudaEvent_t e, unsigned flags) { return (void)s, (void)e, (void)flags, cudaSuccess; }
cudaError_t cudaEventCreateWithFlags(cudaEvent_t *e, unsigned flags) { return (void)flags, *e = NULL, cudaSuccess; }
cudaError_t cudaEventDestroy(cudaEvent_t e) { return (void)e, cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t e, cudaStream_t s) { return (void)e, (void)s, cudaSuccess; }
cudaError_t cudaEventSynchronize(cudaEvent_t e) { return (void)e, cudaSuccess; }
