// Host check of allow_dynamic_smem against a fake runtime of several devices: the
// attribute is set once on each device that launches, again after a failure, and for
// every kernel by itself.  Prints "ok" and exits 0, or the first disagreement and exits 1.
#include <cstdio>
#include <map>
#include <utility>

#include "sg_smem.h"

static int g_device = 0;
static cudaError_t g_next = cudaSuccess;
static std::map<std::pair<int, const void*>, int> g_calls, g_bytes;

extern "C" cudaError_t CUDARTAPI cudaGetDevice(int* device) {
  *device = g_device;
  return cudaSuccess;
}
extern "C" cudaError_t CUDARTAPI cudaFuncSetAttribute(const void* f, cudaFuncAttribute attr, int value) {
  if (attr != cudaFuncAttributeMaxDynamicSharedMemorySize) return cudaErrorInvalidValue;
  ++g_calls[{g_device, f}];
  if (g_next == cudaSuccess) g_bytes[{g_device, f}] = value;
  return g_next;
}

#define EXPECT(x) \
  if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }

int main() {
  const int a = 0, b = 0;
  sg::DeviceBits da{0}, db{0};
  for (int round = 0; round < 3; ++round)
    for (int dev : {0, 1, 7, 63}) {
      g_device = dev;
      EXPECT(sg::allow_dynamic_smem(&a, 230000, &da) == cudaSuccess);
      EXPECT((g_calls[{dev, &a}] == 1 && g_bytes[{dev, &a}] == 230000));
    }
  g_device = 1;
  g_next = cudaErrorInvalidValue;
  EXPECT(sg::allow_dynamic_smem(&b, 100000, &db) == cudaErrorInvalidValue);
  g_next = cudaSuccess;
  EXPECT(sg::allow_dynamic_smem(&b, 100000, &db) == cudaSuccess);
  EXPECT(sg::allow_dynamic_smem(&b, 100000, &db) == cudaSuccess);
  EXPECT((g_calls[{1, &b}] == 2 && g_bytes[{1, &b}] == 100000));
  EXPECT((g_calls.count({0, &b}) == 0));
  std::printf("ok\n");
  return 0;
}
