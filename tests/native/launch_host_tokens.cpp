// The host side of the seam, embedding and AdamW calls over a stand-in for the HIP
// runtime that launches nothing: it checks each launch against the card's limits
// and refuses it as the runtime does.  Reads one call a line from stdin,
//   seam rows cols dtype gate | seam_grad rows cols dtype gate |
//   embed tokens vocab cols dtype | embed_grad tokens vocab cols dtype accumulate |
//   adamw count n bits
// and prints the workspace's or plan's bytes, the status and the number of launches
// (AdamW's: the norm's and the step's).

#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstdio>
#include <cstring>
#include <iostream>
#include <sstream>
#include <string>
#include <vector>

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
  std::string line, what;
  while (std::getline(std::cin, line)) {
    std::istringstream in(line);
    in >> what;
    int64_t a[5] = {0, 0, 0, 0, 0}, bytes = 0;
    for (auto &v : a) in >> v;
    int rc = -100;
    launches = 0;
    if (what == "seam" || what == "seam_grad") {
      zs_blocknorm_desc d{};
      d.rows = a[0];
      d.cols = a[1];
      d.dtype = int32_t(a[2]);
      d.param_dtype = ZS_F32;
      d.kind = ZS_NORM_LAYER;
      d.post = 1;
      d.gate = int32_t(a[3]);
      d.eps = 1e-5f;
      d.residual_scale = 1.0f;
      void *gate = d.gate == ZS_GATE_NONE ? nullptr : at(3);
      void *dgate = d.gate == ZS_GATE_NONE ? nullptr : at(4);
      bytes = zero_shard_blocknorm_workspace(&d);
      if (what == "seam")
        rc = zero_shard_blocknorm(&d, at(1), at(2), gate, at(5), at(6), at(7), at(8), at(9), at(10),
                                  f32(11));
      else
        rc = zero_shard_blocknorm_bwd(&d, at(1), at(2), at(9), at(10), gate, at(5), at(6), at(7),
                                      f32(11), at(12), at(13), dgate, at(14), at(15), at(16),
                                      at(17), at(18), bytes);
    } else if (what == "embed" || what == "embed_grad") {
      zs_embedding_desc d{};
      d.tokens = a[0];
      d.vocab = a[1];
      d.cols = a[2];
      d.dtype = d.table_dtype = d.grad_dtype = int32_t(a[3]);
      d.accumulate = int32_t(a[4]);
      d.id_bytes = 8;
      d.scale = 1.0f;
      bytes = zero_shard_embedding_workspace(&d);
      rc = what == "embed" ? zero_shard_embedding(&d, at(1), at(2), at(3))
                           : zero_shard_embedding_bwd(&d, at(1), at(2), at(3), at(4), bytes);
    } else if (what == "adamw") {
      zs_adamw_desc d{};
      d.count = a[0];
      d.beta1 = 0.9f;
      d.beta2 = 0.999f;
      d.eps = 1e-8f;
      d.bias_correction = 1;
      d.max_norm = 1.0f;
      std::vector<zs_adamw_tensor> tensors(a[0]);
      std::vector<const void *> grads(a[0], at(9));
      uintptr_t next = uintptr_t(1) << 44;
      const auto take = [&](int64_t size) {
        const uintptr_t p = next;
        next += uintptr_t(size + 255) / 256 * 256;
        return reinterpret_cast<void *>(p);
      };
      for (auto &t : tensors) {
        t = zs_adamw_tensor{};
        t.n = a[1];
        t.state = a[2] == 8 ? ZS_STATE_8 : ZS_STATE_32;
        t.grad_dtype = t.param_dtype = ZS_BF16;
        t.lr_scale = 1.0f;
        const int64_t size = a[2] == 8 ? 1 : 4, scales = (t.n + 255) / 256 * 4;
        t.master_out = static_cast<float *>(take(4 * t.n));
        t.master_in = t.master_out;
        t.m_in = t.m_out = take(size * t.n);
        t.v_in = t.v_out = take(size * t.n);
        t.param_out = take(2 * t.n);
        if (a[2] == 8) {
          t.m_scale_in = t.m_scale_out = static_cast<float *>(take(scales));
          t.v_scale_in = t.v_scale_out = static_cast<float *>(take(scales));
        }
      }
      bytes = zero_shard_adamw_plan_bytes(&d, tensors.data());
      rc = bytes < 0 ? ZS_EINVAL : ZS_OK;
      if (rc == ZS_OK) {
        std::vector<uint64_t> plan(size_t(bytes) / 8 + 2);
        void *host = reinterpret_cast<void *>((uintptr_t(plan.data()) + 15) / 16 * 16);
        rc = zero_shard_adamw_plan(&d, tensors.data(), host, bytes);
        if (rc == ZS_OK)
          rc = zero_shard_adamw_gnorm(&d, host, at(3), grads.data(), static_cast<double *>(at(4)));
        if (rc == ZS_OK)
          rc = zero_shard_adamw(&d, host, at(3), grads.data(), 1e-3f, 1, 1,
                                static_cast<const double *>(at(4)));
      }
    }
    std::printf("%s: %lld %d %d\n", line.c_str(), static_cast<long long>(bytes), rc, launches);
  }
  return 0;
}
