// The host side of the layer-norm and Muon calls over a stand-in for the HIP
// runtime that launches nothing: it checks each launch against the card's limits
// and refuses it as the runtime does.  Reads one call a line from stdin,
//   ortho batch rows cols dtype steps | norm rows cols dtype |
//   norm_grad rows cols dtype | momentum n n_d dtype | apply n
// and prints the workspace's bytes, the status and the number of launches.

#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstdio>
#include <cstring>
#include <iostream>
#include <sstream>
#include <string>

#include "zero_shard.h"

namespace {
dim3 grid_, block_;
int launches;
hipError_t last = hipSuccess;

bool fits(unsigned grid, unsigned block, unsigned most) {
  return grid >= 1 && grid <= most && uint64_t(grid) * block <= UINT32_MAX;
}
}  // namespace

extern "C" {
hipError_t hipGetDevice(int *d) {
  *d = 0;
  return hipSuccess;
}
hipError_t hipGetDeviceProperties(hipDeviceProp_t *p, int) {
  std::memset(p, 0, sizeof *p);
  std::strcpy(p->gcnArchName, "gfx950");
  return hipSuccess;
}
hipError_t hipGetLastError() {
  const hipError_t e = last;
  last = hipSuccess;
  return e;
}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t, hipStream_t) {
  grid_ = grid;
  block_ = block;
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3 *grid, dim3 *block, size_t *shared, hipStream_t *stream) {
  *grid = grid_;
  *block = block_;
  *shared = 0;
  *stream = nullptr;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void *, dim3 grid, dim3 block, void **, size_t, hipStream_t) {
  ++launches;
  if (!fits(grid.x, block.x, 0x7fffffff) || !fits(grid.y, block.y, 65535) ||
      !fits(grid.z, block.z, 65535) || uint64_t(block.x) * block.y * block.z > 1024)
    last = hipErrorInvalidConfiguration;
  return last;
}
void **__hipRegisterFatBinary(const void *) { return nullptr; }
void __hipUnregisterFatBinary(void **) {}
void __hipRegisterFunction(void **, const void *, char *, const char *, unsigned, void *, void *,
                           void *, void *, int *) {}
}

int main() {
  // stand-in addresses, aligned and never read
  const auto at = [](uintptr_t i) { return reinterpret_cast<void *>(i << 44); };
  const auto f32 = [&](uintptr_t i) { return static_cast<float *>(at(i)); };
  const auto u16 = [&](uintptr_t i) { return static_cast<uint16_t *>(at(i)); };
  const uint16_t *rows_of[ZS_MAX_ND];
  for (auto &r : rows_of) r = u16(4);
  std::string line, what;
  while (std::getline(std::cin, line)) {
    std::istringstream in(line);
    in >> what;
    int64_t a[5] = {0, 0, 0, 0, 0}, bytes = 0;
    for (int64_t &v : a) in >> v;
    int rc = 0;
    launches = 0;
    if (what == "ortho") {
      zs_ortho_desc d = {};
      d.batch = a[0], d.rows = a[1], d.cols = a[2];
      d.dtype = int32_t(a[3]), d.steps = int32_t(a[4]), d.eps = 1e-7f;
      bytes = zero_shard_ortho_workspace(&d);
      rc = zero_shard_ortho(&d, at(1), u16(2), at(3), bytes);
    } else if (what == "norm" || what == "norm_grad") {
      zs_layernorm_desc d = {};
      d.rows = a[0], d.cols = a[1];
      d.dtype = d.param_dtype = int32_t(a[2]), d.eps = 1e-5f;
      bytes = zero_shard_layernorm_workspace(&d);
      rc = what == "norm" ? zero_shard_layernorm(&d, at(1), nullptr, at(4), at(5), nullptr, at(1),
                                                 f32(6), f32(7))
                          : zero_shard_layernorm_bwd(&d, at(1), at(2), at(4), f32(6), f32(7),
                                                     nullptr, at(1), at(5), at(8), at(3), bytes);
    } else {
      zs_muon_desc d = {};
      d.n = a[0], d.n_d = what == "momentum" ? int32_t(a[1]) : 1;
      d.dtype = int32_t(a[2]), d.mu = 0.95f;
      rc = what == "momentum"
               ? zero_shard_muon_momentum(&d, rows_of, f32(1), f32(1), at(2))
               : zero_shard_muon_apply(&d, u16(2), 0.1f, 1.0f, f32(1), f32(1), u16(3));
    }
    std::printf("%s: %lld %d %d\n", line.c_str(), static_cast<long long>(bytes), rc, launches);
  }
  return 0;
}
