// A HIP runtime that launches nothing: it writes down the kernels that a library
// registers, the limits on their dynamic LDS and the launches (test_launches_cpu.py).
#include <cstddef>
#include <cstdio>

struct Dim3 { unsigned x, y, z; };
struct Config { Dim3 grid, block; size_t lds; void* stream; };
static Config pushed;

extern "C" {
void** __hipRegisterFatBinary(const void*) { static void* module; return &module; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
void __hipRegisterFunction(void**, const void* f, char*, const char* name, unsigned, void*, void*, Dim3*, Dim3*, int*) {
  std::printf("kernel %p %s\n", f, name);
}
int __hipPushCallConfiguration(Dim3 grid, Dim3 block, size_t lds, void* stream) {
  pushed = Config{grid, block, lds, stream};
  return 0;
}
int __hipPopCallConfiguration(Dim3* grid, Dim3* block, size_t* lds, void** stream) {
  *grid = pushed.grid, *block = pushed.block, *lds = pushed.lds, *stream = pushed.stream;
  return 0;
}
int hipLaunchKernel(const void* f, Dim3 grid, Dim3 block, void**, size_t lds, void*) {
  std::printf("launch %p %zu %u %u %u %u\n", f, lds, grid.x, grid.y, grid.z, block.x * block.y * block.z);
  return 0;
}
int hipFuncSetAttribute(const void* f, int, int value) {
  std::printf("limit %p %d\n", f, value);
  return 0;
}
int hipGetLastError() { return 0; }
int hipGetDevice(int* device) { return *device = 0; }
int hipDeviceGetAttribute(int* value, int, int) { *value = 256; return 0; }
int hipGetSymbolAddress(void** address, const void*) { *address = nullptr; return 1; }
}
