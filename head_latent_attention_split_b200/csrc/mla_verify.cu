// Verification of drafted tokens against the target's probabilities (mla_verify_drafts in
// include/mla_decode.h): the accepted prefix, one token drawn from the residual by inverse
// CDF, and the sequence's new length.
//
// Only one row of each distribution is read, the one behind the last accepted draft, so a sequence
// costs 2 V values. A cluster of C CTAs shares it. The row is cut into chunks of 512
// values; a warp sums a chunk (16 weights per lane, all loads issued together) and the chunk
// sums stay in shared memory. One exchange of the CTAs' sums gives the total, the draw's target
// and the CTA that holds it, which finds the chunk among its sums and reads that chunk again.
// All sums are fp64: the weights are fp32 or bf16 and the draw has to fall on the same token
// whatever the order of the sum, so its rounding must be far below a weight. Every CTA adds in the
// same order (chunk, prefix of chunks, prefix of CTAs): the result does not vary between runs.
#include "mla_device.cuh"
#include "ptx_sm100.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kVfThreads = 256;
constexpr int kVfWarps = kVfThreads / 32;
constexpr int kVfChunk = 512;          // values per chunk
constexpr int kVfPer = kVfChunk / 32;  // per lane
constexpr int kVfMaxCluster = 8;
constexpr int kVfMaxChunks = 2048;     // per CTA; V <= 2048 * 512 * 8 = 8 Mi

struct VerifyArgs {
  int B, K, V;
  const void* target;          // [B, K + 1, V]
  const void* draft;           // [B, K, V] or null
  const int32_t* tokens;       // [B, K]
  const int32_t* lens;         // [B] or null
  const float* accept_u;       // [B, K]
  const float* sample_u;       // [B]
  const int32_t* seq_lens;     // [B] or null
  int32_t* out;                // [B, K + 1]
  int32_t* accepted;           // [B]
  int32_t* new_seq_lens;       // [B] or null
  int* status;
};

__device__ __forceinline__ float prob(const float* p, size_t i) { return __ldg(p + i); }
__device__ __forceinline__ float prob(const uint16_t* p, size_t i) { return bf16_bits_to_float(__ldg(p + i)); }

__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ double warp_scan64(double v) {   // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

__device__ __forceinline__ double ld_cluster_f64(uint32_t addr) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
  return v;
}

// The weight of a token: max(p - q, 0); not above 0 (NaN included) counts as 0.
__device__ __forceinline__ double weight(float p, float q) {
  const double w = (double)p - (double)q;
  return w > 0.0 ? w : 0.0;
}

// kVec: rows are whole 16-byte pieces (V a multiple of the values per piece, 16-byte aligned bases)
template <typename T, bool kVec>
__global__ void __launch_bounds__(kVfThreads, 4) verify_kernel(const VerifyArgs a) {
  constexpr int kPiece = 16 / (int)sizeof(T);
  __shared__ double chunk_sum[kVfMaxChunks];
  __shared__ double part[2];      // this CTA's sum, one slot per pass
  __shared__ int s_n, s_tok;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t C, rank = cluster_ctarank();
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
  const int b = blockIdx.x / C;
  const int K = a.K, V = a.V;
  const T* target = (const T*)a.target + (size_t)b * (K + 1) * V;
  const T* draft = a.draft ? (const T*)a.draft + (size_t)b * K * V : nullptr;
  const int nd_raw = a.lens ? __ldg(a.lens + b) : K;
  const bool bad_len = nd_raw < 0 || nd_raw > K;
  const int nd = bad_len ? 0 : nd_raw;

  if (warp == 0) {
    // the first draft that is refused; s_n = -1: its token id cannot be used
    int n = nd, tok = -1;
    for (int i0 = 0; i0 < nd; i0 += 32) {
      const int i = i0 + lane;
      bool stop = false, bad = false;
      int x = -1;
      if (i < nd) {
        x = __ldg(a.tokens + (size_t)b * K + i);
        bad = x < 0 || x >= V;
        stop = true;
        if (!bad) {
          const double p = prob(target, (size_t)i * V + x);
          const double q = draft ? (double)prob(draft, (size_t)i * V + x) : 1.0;
          stop = !((double)__ldg(a.accept_u + (size_t)b * K + i) * q < p);   // exact in fp64; NaN refuses
        }
      }
      const unsigned m = __ballot_sync(0xffffffffu, stop);
      if (m) {
        const int src = __ffs(m) - 1;
        n = __shfl_sync(0xffffffffu, bad, src) ? -1 : i0 + src;
        tok = __shfl_sync(0xffffffffu, x, src);
        break;
      }
    }
    if (lane == 0) {
      s_n = n;
      s_tok = tok;
    }
  }
  __syncthreads();
  int n = s_n;
  const int tok = s_tok;   // the refused draft (draft null: its weight is 0)
  bool bad = bad_len || n < 0;
  int got = -1;

  if (!bad) {   // the same branch in every CTA of the cluster
    const T* p = target + (size_t)n * V;
    const bool refused = n < nd;
    const T* q = refused && draft ? draft + (size_t)n * V : nullptr;
    const int chunks = (V + kVfChunk - 1) / kVfChunk;
    const int c0 = (int)((long long)chunks * rank / C), c1 = (int)((long long)chunks * (rank + 1) / C);
    float u = __ldg(a.sample_u + b);
    u = u >= 1.f ? 0x1.fffffep-1f : u >= 0.f ? u : 0.f;
    double before = 0.0, total = 0.0;
    bool residual = refused;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      // pass 1 only when the residual is 0 everywhere: the target's own row
      const T* qq = residual ? q : nullptr;
      const int hole = residual && !draft ? tok : -1;
      for (int c = c0 + warp; c < c1; c += kVfWarps) {
        const int base = c * kVfChunk;
        double s = 0.0;
        if constexpr (kVec) {
          constexpr int kLoads = kVfPer / kPiece;
          uint4 pv[kLoads], qv[kLoads];
#pragma unroll
          for (int l = 0; l < kLoads; ++l) {
            const int i = base + (32 * l + lane) * kPiece;
            pv[l] = qv[l] = make_uint4(0u, 0u, 0u, 0u);
            if (i < V) {
              pv[l] = __ldg(reinterpret_cast<const uint4*>(p + i));
              if (qq) qv[l] = __ldg(reinterpret_cast<const uint4*>(qq + i));
            }
          }
#pragma unroll
          for (int l = 0; l < kLoads; ++l) {
            const int i = base + (32 * l + lane) * kPiece;
            const uint32_t pw[4] = {pv[l].x, pv[l].y, pv[l].z, pv[l].w}, qw[4] = {qv[l].x, qv[l].y, qv[l].z, qv[l].w};
#pragma unroll
            for (int e = 0; e < kPiece; ++e) {
              float x, y;
              if constexpr (sizeof(T) == 4) {
                x = __uint_as_float(pw[e]);
                y = __uint_as_float(qw[e]);
              } else {
                x = __uint_as_float(e & 1 ? pw[e >> 1] & 0xFFFF0000u : pw[e >> 1] << 16);
                y = __uint_as_float(e & 1 ? qw[e >> 1] & 0xFFFF0000u : qw[e >> 1] << 16);
              }
              s += i + e == hole ? 0.0 : weight(x, y);
            }
          }
        } else {
          float x[kVfPer], y[kVfPer];
#pragma unroll
          for (int e = 0; e < kVfPer; ++e) {
            const int i = base + 32 * e + lane;
            x[e] = i < V ? prob(p, i) : 0.f;
            y[e] = i < V && qq ? prob(qq, i) : 0.f;
          }
#pragma unroll
          for (int e = 0; e < kVfPer; ++e) s += base + 32 * e + lane == hole ? 0.0 : weight(x[e], y[e]);
        }
        s = warp_sum64(s);
        if (lane == 0) chunk_sum[c - c0] = s;
      }
      __syncthreads();
      if (warp == 0) {
        // inclusive prefix of the chunk sums in place; the CTA's sum
        double run = 0.0;
        for (int i0 = 0; i0 < c1 - c0; i0 += 32) {
          const int i = i0 + lane;
          const double v = warp_scan64(i < c1 - c0 ? chunk_sum[i] : 0.0) + run;
          if (i < c1 - c0) chunk_sum[i] = v;
          run = __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) part[pass] = run;
      }
      if (C > 1) cluster_sync(); else __syncthreads();
      before = total = 0.0;
      for (uint32_t r = 0; r < C; ++r) {
        const double v = C == 1 ? part[pass] : ld_cluster_f64(mapa(smem_u32(&part[pass]), r));
        if (r == rank) before = total;
        total += v;
      }
      if (total > 0.0 || !residual) break;
      residual = false;
    }
    bad = !(total > 0.0 && total <= 1.7976931348623157e308);
    const double goal = (double)u * total;
    // the CTA whose range [before, before + own sum) holds the goal; the same additions in every CTA
    const bool mine = !bad && before <= goal && goal < before + part[residual || !refused ? 0 : 1];
    if (mine && warp == 0) {
      int lo = 0, hi = c1 - c0 - 1;   // first chunk whose prefix exceeds the goal
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (before + chunk_sum[mid] > goal) hi = mid; else lo = mid + 1;
      }
      double run = before + (lo > 0 ? chunk_sum[lo - 1] : 0.0);
      const int base = (c0 + lo) * kVfChunk + lane * kVfPer;   // 16 consecutive values per lane
      const T* qq = residual ? q : nullptr;
      const int hole = residual && !draft ? tok : -1;
      double w[kVfPer], s = 0.0;
#pragma unroll
      for (int e = 0; e < kVfPer; ++e) {
        const int i = base + e;
        w[e] = i < V && i != hole ? weight(prob(p, i), qq ? prob(qq, i) : 0.f) : 0.0;
        s += w[e];
      }
      const double upto = run + warp_scan64(s);
      run = upto - s;
      int at = -1, last = -1;   // first value past the goal; last one with a weight
#pragma unroll
      for (int e = 0; e < kVfPer; ++e) {
        run += w[e];
        if (w[e] > 0.0) {
          last = base + e;
          if (at < 0 && run > goal) at = base + e;
        }
      }
      const unsigned hit = __ballot_sync(0xffffffffu, at >= 0), any = __ballot_sync(0xffffffffu, last >= 0);
      // (the sums inside the chunk round differently from its prefix: without a hit, its last weight)
      got = hit ? __shfl_sync(0xffffffffu, at, __ffs(hit) - 1)
                : __shfl_sync(0xffffffffu, last, any ? 31 - __clz(any) : 0);
      if (lane == 0) a.out[(size_t)b * (K + 1) + n] = got;
    }
  }
  if (rank == 0) {
    for (int i = tid; i <= K; i += kVfThreads) {
      if (bad || i > n)
        a.out[(size_t)b * (K + 1) + i] = -1;
      else if (i < n)
        a.out[(size_t)b * (K + 1) + i] = __ldg(a.tokens + (size_t)b * K + i);
    }
    if (tid == 0) {
      if (bad) set_status(a.status, MLA_ERR_BAD_INPUT);
      a.accepted[b] = bad ? -1 : n;
      if (a.new_seq_lens) a.new_seq_lens[b] = __ldg(a.seq_lens + b) - nd + (bad ? 0 : n);
    }
  }
  if (C > 1) cluster_sync();   // no CTA leaves while a peer may still read its sum
}

template <typename T>
cudaError_t launch(const VerifyArgs& a, bool vec, int C, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.B * C));
  cfg.blockDim = dim3(kVfThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)C;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return vec ? cudaLaunchKernelEx(&cfg, verify_kernel<T, true>, a) : cudaLaunchKernelEx(&cfg, verify_kernel<T, false>, a);
}

}  // namespace
}  // namespace mla

extern "C" mla_status_t mla_verify_drafts(const mla_verify_params_t* p, const void* target, const void* draft,
                                          const int32_t* draft_tokens, const int32_t* draft_lens,
                                          const float* accept_u, const float* sample_u, const int32_t* seq_lens,
                                          int32_t* tokens, int32_t* accepted, int32_t* new_seq_lens, void* stream) {
  using namespace mla;
  if (!p || p->batch < 0 || p->max_drafts < 0 || p->vocab < 1 || p->reserved != 0 ||
      (p->prob_dtype != MLA_DTYPE_F32 && p->prob_dtype != MLA_DTYPE_BF16))
    return MLA_ERR_INVALID_ARG;
  if (p->vocab > kVfMaxChunks * kVfChunk * kVfMaxCluster || p->batch > (1 << 27) || p->max_drafts > (1 << 20))
    return MLA_ERR_UNSUPPORTED;
  if (p->batch == 0) return MLA_OK;
  if (!target || !sample_u || !tokens || !accepted || (p->max_drafts > 0 && (!draft_tokens || !accept_u)))
    return MLA_ERR_INVALID_ARG;
  if ((seq_lens == nullptr) != (new_seq_lens == nullptr)) return MLA_ERR_INVALID_ARG;
  const size_t e = p->prob_dtype == MLA_DTYPE_F32 ? 4 : 2;
  if ((uintptr_t)target % e || (uintptr_t)draft % e) return MLA_ERR_ALIGNMENT;
  const void* p4[] = {draft_tokens, draft_lens, accept_u, sample_u, seq_lens, tokens, accepted, new_seq_lens};
  for (const void* q : p4)
    if ((uintptr_t)q % 4) return MLA_ERR_ALIGNMENT;
  int* status = current_status_word();
  if (!status) return MLA_ERR_CUDA;
  const VerifyArgs a{p->batch, p->max_drafts, p->vocab, target, draft, draft_tokens, draft_lens, accept_u, sample_u,
                     seq_lens, tokens, accepted, new_seq_lens, status};
  const bool vec = (size_t)p->vocab * e % 16 == 0 && ((uintptr_t)target | (uintptr_t)draft) % 16 == 0;
  // CTAs per sequence: one per 4096 values (the loads that 8 warps issue at once), up to 8, but no more
  // than it takes to give every SM its four: a longer slice hides the chain of dependent loads before it
  int dev = 0, sms = 0, C = 1;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MLA_ERR_CUDA;
  while (C < kVfMaxCluster && (int64_t)C * 4096 < p->vocab && (int64_t)p->batch * C < 4 * sms) C *= 2;
  // (a slice's chunk sums have to fit)
  while (C < kVfMaxCluster && (int64_t)C * kVfMaxChunks * kVfChunk < p->vocab) C *= 2;
  const cudaError_t err = e == 4 ? launch<float>(a, vec, C, (cudaStream_t)stream)
                                 : launch<uint16_t>(a, vec, C, (cudaStream_t)stream);
  return err == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
