// Verification of drafted tokens against the target's probabilities (mla_verify_drafts in
// include/mla_decode.h): the accepted prefix, one token drawn from the residual by inverse
// CDF, and the sequence's new length.
//
// Only one row of each distribution is read, the one behind the last accepted draft, so a sequence
// costs 2 V values. A cluster of C CTAs shares it. The row is cut into chunks of 1024
// values; a warp sums a chunk (32 weights per lane, the next 8 pairs on their way while 8 are added)
// and the chunk sums stay in shared memory. One exchange of the CTAs' sums gives the total, the draw's target
// and the CTA that holds it, which finds the chunk among its sums and reads that chunk again.
// All sums are fp64: the weights are fp32 or bf16 and the draw has to fall on the same token
// whatever the order of the sum, so its rounding must be far below a weight. Every CTA adds in the
// same order (chunk, prefix of chunks, prefix of CTAs): the result does not vary between runs.
// Bound: the reads where the batch is large (128 sequences of 128000 fp32 values in 28 us, 4.7 TB/s;
// conversions and fp64 sums keep 44 % of the issue slots busy), the chain of dependent loads where it
// is small (one sequence of 32000 in 11 us of device time).
#include <type_traits>

#include "mla_device.cuh"
#include "ptx_sm100.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kVfThreads = 256;
constexpr int kVfWarps = kVfThreads / 32;
constexpr int kVfChunk = 1024;         // values per chunk
constexpr int kVfPer = kVfChunk / kVfThreads;   // per thread when a chunk is searched
constexpr int kNone = 0x7fffffff;
constexpr double kMaxDouble = 1.7976931348623157e308;
constexpr int kVfMaxCluster = 8;
constexpr int kVfMaxChunks = 1024;     // per CTA; V <= 1024 * 1024 * 8 = 8 Mi

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

// One lane's part of kCount = 32 x kPer consecutive values of a row pair: loaded, then added.
// kVec: rows are whole 16-byte pieces (V a multiple of the values per piece, 16-byte aligned bases).
template <typename T, bool kVec>
struct Unit {
  static constexpr int kPiece = kVec ? 16 / (int)sizeof(T) : 1, kLoads = kVec ? 2 : 8;
  static constexpr int kCount = 32 * kPiece * kLoads;
  typedef typename std::conditional<kVec, uint4, T>::type Word;
  Word p[kLoads], q[kLoads];

  __device__ __forceinline__ void load(const T* pr, const T* qr, int base, int V) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      const int i = base + (32 * l + lane) * kPiece;
      p[l] = q[l] = Word();
      if (i < V) {
        p[l] = __ldg(reinterpret_cast<const Word*>(pr + i));
        if (qr) q[l] = __ldg(reinterpret_cast<const Word*>(qr + i));
      }
    }
  }
  static __device__ __forceinline__ float value(const Word& w, int e) {
    if constexpr (kVec) {
      const uint32_t x = (e * (int)sizeof(T)) / 4 == 0 ? w.x : (e * (int)sizeof(T)) / 4 == 1 ? w.y
                         : (e * (int)sizeof(T)) / 4 == 2 ? w.z : w.w;
      return __uint_as_float(sizeof(T) == 4 ? x : e & 1 ? x & 0xFFFF0000u : x << 16);
    } else if constexpr (sizeof(T) == 4) {
      return w;
    } else {
      return bf16_bits_to_float(w);
    }
  }
  // Two running sums, for the length of the chain of additions. kCareful: as weight() says, and
  // without the token `hole`; otherwise max(p, q) - q, the same number for finite p and q (and
  // NaN or an infinity in the sum where they are not).
  template <bool kCareful>
  __device__ __forceinline__ void add(double& s0, double& s1, int base, int hole) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      const int i = base + (32 * l + lane) * kPiece;
#pragma unroll
      for (int e = 0; e < kPiece; ++e) {
        const float x = value(p[l], e), y = value(q[l], e);
        const double w = kCareful ? (i + e == hole ? 0.0 : weight(x, y)) : (double)fmaxf(x, y) - (double)y;
        if ((l * kPiece + e) & 1) s1 += w; else s0 += w;
      }
    }
  }
};

template <typename T, bool kVec>
__global__ void __launch_bounds__(kVfThreads, 4) verify_kernel(const VerifyArgs a) {
  __shared__ double chunk_sum[kVfMaxChunks];
  __shared__ double part[3];      // this CTA's sum, one slot per pass
  __shared__ double warp_sum[kVfWarps];
  __shared__ int s_n, s_tok, s_at, s_last;
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
      s_at = kNone;
      s_last = -1;
    }
  }
  __syncthreads();
  int n = s_n;
  const int tok = s_tok;   // the refused draft (draft null: its weight is 0)
  bool bad = bad_len || n < 0;

  if (!bad) {   // the same branch in every CTA of the cluster
    const T* p = target + (size_t)n * V;
    const bool refused = n < nd;
    const T* q = refused && draft ? draft + (size_t)n * V : nullptr;
    const int chunks = (V + kVfChunk - 1) / kVfChunk;
    const int c0 = (int)((long long)chunks * rank / C), c1 = (int)((long long)chunks * (rank + 1) / C);
    float u = __ldg(a.sample_u + b);
    u = u >= 1.f ? 0x1.fffffep-1f : u >= 0.f ? u : 0.f;
    double before = 0.0, total = 0.0;
    bool residual = refused, careful = false;
    int pass = 0;
#pragma unroll 1
    for (;; ++pass) {
      // One pass, as a rule. Again with care when the sum is not finite; again over the target's own row
      // when the residual is 0 everywhere: three at most.
      const T* qq = residual ? q : nullptr;
      const int hole = residual && !draft ? tok : -1;
      // this warp's chunks as one stream of units, the next one loading while one is added
      typedef Unit<T, kVec> U;
      constexpr int kUnits = kVfChunk / U::kCount;
      const int mine_chunks = c0 + warp < c1 ? (c1 - c0 - warp + kVfWarps - 1) / kVfWarps : 0;
      auto unit_base = [&](int i) { return (c0 + warp + (i / kUnits) * kVfWarps) * kVfChunk + (i % kUnits) * U::kCount; };
      U buf[2];
      double sa = 0.0, sb = 0.0;
      if (mine_chunks > 0) buf[0].load(p, qq, unit_base(0), V);
#pragma unroll 1
      for (int i = 0; i < mine_chunks * kUnits; i += 2) {   // kUnits is even
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (i + h + 1 < mine_chunks * kUnits) buf[h ^ 1].load(p, qq, unit_base(i + h + 1), V);
          const int ub = unit_base(i + h);
          if (careful || (hole >= ub && hole < ub + U::kCount))
            buf[h].template add<true>(sa, sb, ub, hole);
          else
            buf[h].template add<false>(sa, sb, ub, hole);
        }
        if ((i + 2) % kUnits == 0) {
          const double s = warp_sum64(sa + sb);
          if (lane == 0) chunk_sum[warp + (i / kUnits) * kVfWarps] = s;
          sa = sb = 0.0;
        }
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
      if (!careful && !(total <= kMaxDouble)) {
        careful = true;
      } else if (total > 0.0 || !residual) {
        break;
      } else {
        residual = false;
      }
    }
    bad = !(total > 0.0 && total <= kMaxDouble);
    const double goal = (double)u * total;
    // the CTA whose range [before, before + own sum) holds the goal; the same additions in every CTA
    const bool mine = !bad && before <= goal && goal < before + part[pass];
    if (mine) {   // the whole block: one chunk, four consecutive values per thread
      int lo = 0, hi = c1 - c0 - 1;   // first chunk whose prefix exceeds the goal
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (before + chunk_sum[mid] > goal) hi = mid; else lo = mid + 1;
      }
      const double run = before + (lo > 0 ? chunk_sum[lo - 1] : 0.0);
      const int base = (c0 + lo) * kVfChunk + tid * kVfPer;
      const T* qq = residual ? q : nullptr;
      const int hole = residual && !draft ? tok : -1;
      double w[kVfPer], s = 0.0;
#pragma unroll
      for (int e = 0; e < kVfPer; ++e) {
        const int i = base + e;
        w[e] = i < V && i != hole ? weight(prob(p, i), qq ? prob(qq, i) : 0.f) : 0.0;
        s += w[e];
      }
      const double incl = warp_scan64(s);
      if (lane == 31) warp_sum[warp] = incl;
      __syncthreads();
      double upto = run;
      for (int i = 0; i < warp; ++i) upto += warp_sum[i];
      upto += incl - s;
      int at = kNone, last = -1;   // first value past the goal; last one with a weight
#pragma unroll
      for (int e = 0; e < kVfPer; ++e) {
        upto += w[e];
        if (w[e] > 0.0) {
          last = base + e;
          if (at == kNone && upto > goal) at = base + e;
        }
      }
      at = __reduce_min_sync(0xffffffffu, at);
      last = __reduce_max_sync(0xffffffffu, last);
      if (lane == 0) {
        atomicMin(&s_at, at);
        atomicMax(&s_last, last);
      }
      __syncthreads();
      // (the sums inside the chunk round differently from its prefix: without a hit, its last weight)
      if (tid == 0) a.out[(size_t)b * (K + 1) + n] = s_at != kNone ? s_at : s_last;
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
  // CTAs per sequence: one per 4096 values (what 8 warps load at once), up to 8, but no more than it
  // takes to give every SM two: a longer slice hides the chain of dependent loads before it (128
  // sequences of 128000 values, the weights still summed with their checks: 40 us with 8, 35 us with 4, 41 us
  // with 2; 28 us with 4 since)
  int dev = 0, sms = 0, C = 1;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MLA_ERR_CUDA;
  while (C < kVfMaxCluster && (int64_t)C * 4096 < p->vocab && (int64_t)p->batch * C < 2 * sms) C *= 2;
  // (a slice's chunk sums have to fit)
  while (C < kVfMaxCluster && (int64_t)C * kVfMaxChunks * kVfChunk < p->vocab) C *= 2;
  const cudaError_t err = e == 4 ? launch<float>(a, vec, C, (cudaStream_t)stream)
                                 : launch<uint16_t>(a, vec, C, (cudaStream_t)stream);
  return err == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
