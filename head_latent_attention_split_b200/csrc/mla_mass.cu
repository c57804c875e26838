// Attention weight per cached token (mla_attention_mass in include/mla_decode.h):
//   mass[b, t] = mass_in[b, t] + sum over rows (s, h) that see t of exp(sigma_t(s, h) - lse[b, s, h]).
//
// mass_simt_kernel: fp32 CUDA cores, any width, block size and storage type. A CTA takes 32 tokens
// of one sequence, decoded to fp32 in shared memory; lane = token, a warp takes every eighth group
// of four query rows, so one token value serves four products. Bound by the fp32 products (and the
// shared-memory reads that feed them); it serves the shapes the tensor kernel does not take.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "mla_device.cuh"

namespace mla {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTok = 32;    // tokens per CTA, one per lane
constexpr int kQRows = 4;   // query rows per warp and step

__global__ void __launch_bounds__(kThreads) mass_simt_kernel(const MassArgs m) {
  extern __shared__ float tok[];   // [kTok][D + 1]
  __shared__ float part[kWarps][kTok];
  const DecodeArgs& a = m.d;
  const int D = a.r + a.d_r, ld = D + 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr float kLog2e = 1.4426950408889634f;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const int L = __ldg(a.seq_lens + b);
    if (L < 0 || L > a.len_cap) {
      if (blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, MLA_ERR_BAD_SEQ_LEN);
      continue;
    }
    const int t0 = blockIdx.x * kTok, nt = min(L - t0, kTok);
    if (nt <= 0) continue;
    __syncthreads();
    for (int j = warp; j < nt; j += kWarps) {
      const int t = t0 + j;
      const int blk = __ldg(a.block_table + (size_t)b * a.max_blocks + t / a.bs);
      const bool ok = blk >= 0 && blk < a.num_blocks;
      if (!ok && lane == 0) set_status(a.status, MLA_ERR_BAD_BLOCK_ID);
      const size_t slot = ok ? (size_t)blk * a.bs + t % a.bs : 0;
      for (int k = lane; k < D; k += 32) {
        float v = __uint_as_float(0x7FC00000u);   // a bad block's tokens get NaN
        if (ok) {
          if (a.cache_dtype == kE4M3)
            v = k < a.r ? e4m3_to_float(__ldg((const uint8_t*)a.cache + slot * a.r + k)) * __ldg(a.kv_scale + slot)
                        : bf16_bits_to_float(__ldg(a.k_rope + slot * a.d_r + (k - a.r)));
          else
            v = load_q(a.cache, a.cache_dtype, slot * D + k);
        }
        tok[j * ld + k] = v;
      }
    }
    __syncthreads();
    const float* c = tok + min(lane, nt - 1) * ld;
    const int t = t0 + lane;
    float sum = 0.f;
    for (int r0 = warp * kQRows; r0 < a.rows; r0 += kWarps * kQRows) {
      float d[kQRows];
      size_t row[kQRows];
#pragma unroll
      for (int i = 0; i < kQRows; ++i) {
        d[i] = 0.f;
        row[i] = (size_t)b * a.rows + min(r0 + i, a.rows - 1);
      }
      for (int k = 0; k < a.r; ++k) {
        const float v = c[k];
#pragma unroll
        for (int i = 0; i < kQRows; ++i) d[i] = fmaf(load_q(a.q_lat, a.q_dtype, row[i] * a.r + k), v, d[i]);
      }
      for (int k = 0; k < a.d_r; ++k) {
        const float v = c[a.r + k];
#pragma unroll
        for (int i = 0; i < kQRows; ++i) d[i] = fmaf(load_q(a.q_rope, a.q_dtype, row[i] * a.d_r + k), v, d[i]);
      }
#pragma unroll
      for (int i = 0; i < kQRows; ++i) {
        const int n_row = a.causal ? L - a.Sq + 1 + (r0 + i) / a.H : L;   // tokens this row sees
        if (r0 + i < a.rows && t < n_row) sum += exp2f(fmaf(d[i], a.scale_log2, -__ldg(m.lse + row[i]) * kLog2e));
      }
    }
    part[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && lane < nt) {
      const size_t o = (size_t)b * m.max_seq_len + t;
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) v += part[i][lane];
      m.mass[o] = m.mass_in ? m.mass_in[o] + v : v;
    }
  }
}

}  // namespace

bool mass_tc_supported(int, int, int, int, int) { return false; }
cudaError_t launch_mass_tc(const MassArgs&, cudaStream_t) { return cudaErrorInvalidValue; }

cudaError_t launch_mass_simt(const MassArgs& m, cudaStream_t s) {
  const int smem = kTok * (m.d.r + m.d.d_r + 1) * (int)sizeof(float);
  static std::once_flag once[64];
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t err = cudaSuccess;
  std::call_once(once[dev & 63], [&] {
    err = cudaFuncSetAttribute(mass_simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kTok * (kSimtMaxD + 1) * (int)sizeof(float));
  });
  if (err != cudaSuccess) return err;
  const dim3 grid((unsigned)((m.d.len_cap + kTok - 1) / kTok), (unsigned)std::min(m.d.B, 65535));
  mass_simt_kernel<<<grid, kThreads, smem, s>>>(m);
  return cudaGetLastError();
}

}  // namespace mla
