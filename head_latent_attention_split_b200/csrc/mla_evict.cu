// Eviction from the paged cache by accumulated attention weight: the choice of the tokens that stay
// (mla_evict_select) and their copy into other blocks (mla_cache_compact). See include/mla_decode.h.
//
// Select: of the candidates [sinks, L - recent) of a sequence keep the k = budget - sinks - recent
// largest, ties to the lower position. A radix select in up to three passes (11, 11, 10 bits of an
// order-preserving key; none below a digit whose entries all stay) finds the k-th largest key T and how
// many entries equal to T stay; one prefix sum over (above T, equal to T) counts then places every kept
// position. A thread holds 4, 8 or 16 consecutive keys in registers, so a row is read from memory
// once, and a cluster of C CTAs shares a row of more than 16384 (C <= 8, rounds beyond). Each pass has
// its own histogram, which every CTA sums over the cluster for itself: one cluster barrier per pass.
// A row of a few KB to half a MB is far from any bandwidth: the barriers and the histogram's
// shared-memory atomics bound it. 64 rows of up to 8192 take 11.5 us, one row of 1100 9 us (15.5 us each
// with 16 keys per thread, three passes and six barriers in each).
//
// Compact: a copy, bound by memory: every kept row read and written once. A warp takes 8 entries of
// one sequence; 8 lanes look their slots up and each moves its row by bulk copies through shared
// memory, so the bytes in flight cost no registers (six CTAs of 37 KB per SM for a bf16 row of
// 1152 bytes). 64 sequences of up to 2048 kept rows (126 MB read, as much written): 40 us.
#include <algorithm>
#include <mutex>

#include "mla_device.cuh"
#include "ptx_sm100.cuh"

namespace mla {
namespace {

using namespace ptx;

// ------------------------------------------------------------------------------- select
constexpr int kSelThreads = 1024;
constexpr int kSelPer = 16;                            // consecutive keys per thread, at most
constexpr int kSelMaxCluster = 8;

struct SelectArgs {
  int B, S, budget, sinks, recent;
  const float* mass;         // [B, S]
  const int32_t* seq_lens;   // [B]
  int32_t* indices;          // [B, budget]
  int32_t* counts;           // [B]
  int* status;
};

// order-preserving unsigned key of an fp32 value; -0 and +0 share one, every NaN has the largest
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (x != x) return 0xffffffffu;
  uint32_t u = __float_as_uint(x);
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// Exclusive prefix sum over the block's 1024 threads; *total = the sum. One barrier: every warp sums up
// the 32 warps' totals for itself. wsum is not written again before the block's next barrier but one.
template <class T>
__device__ __forceinline__ T scan_excl(T v, T* wsum, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) wsum[warp] = x;
  __syncthreads();
  T t = wsum[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, t, o);
    if (lane >= o) t += y;
  }
  *total = __shfl_sync(0xffffffffu, t, 31);
  const T before = __shfl_sync(0xffffffffu, t, (warp - 1) & 31);
  return x - v + (warp ? before : (T)0);
}

// kPer: consecutive keys per thread
template <int kPer>
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const SelectArgs a) {
  __shared__ uint32_t hist[3][2048];
  __shared__ uint64_t wsum[2][32];
  __shared__ uint32_t hsum[3][32];
  __shared__ uint32_t pick[3][3];
  __shared__ uint32_t slice[2];   // this CTA's counts of keys above T and equal to T
  launch_dependents();   // the copy
  const int tid = threadIdx.x;
  const uint32_t C = cluster_size(), rank = cluster_ctarank();
  const int b = blockIdx.x / C;
  int L = __ldg(a.seq_lens + b);
  if (L < 0 || L > a.S) {
    if (tid == 0 && rank == 0) set_status(a.status, MLA_ERR_BAD_SEQ_LEN);
    L = 0;
  }
  int32_t* out = a.indices + (size_t)b * a.budget;
  const int step = kSelThreads * (int)C, first = (int)rank * kSelThreads + tid;
  if (tid == 0 && rank == 0) a.counts[b] = min(L, a.budget);
  if (L <= a.budget) {   // everything stays (the same branch in every CTA of the cluster)
    for (int j = first; j < a.budget; j += step) out[j] = j < L ? j : -1;
    return;
  }
  const int k = a.budget - a.sinks - a.recent;   // candidates to keep: fewer than there are
  const int s0 = a.sinks, s1 = L - a.recent;
  for (int j = first; j < a.sinks; j += step) out[j] = j;
  for (int j = first; j < a.recent; j += step) out[a.budget - a.recent + j] = s1 + j;
  if (k == 0) return;

  const float* row = a.mass + (size_t)b * a.S;
  const bool vec = ((uintptr_t)row & 15) == 0;
  // this CTA's positions: rounds of kSpan * C consecutive ones, kSpan per CTA
  constexpr int kSpan = kSelThreads * kPer;
  const int lo = (int)rank * kSpan + tid * kPer;
  const int round = kSpan * (int)C;
  const bool once = s1 <= round;
  uint32_t key[kPer];
  uint32_t in = 0;   // bit m: position p0 + m is a candidate
  auto load = [&](int p0) {
    in = 0;
#pragma unroll
    for (int m = 0; m < kPer; ++m) in |= (p0 + m >= s0 && p0 + m < s1) ? 1u << m : 0u;
#pragma unroll
    for (int m = 0; m < kPer; m += 4) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (vec && p0 + m + 4 <= a.S) {
        if ((in >> m) & 15u) v = __ldg(reinterpret_cast<const float4*>(row + p0 + m));
      } else {
        if ((in >> m) & 1u) v.x = __ldg(row + p0 + m);
        if ((in >> m) & 2u) v.y = __ldg(row + p0 + m + 1);
        if ((in >> m) & 4u) v.z = __ldg(row + p0 + m + 2);
        if ((in >> m) & 8u) v.w = __ldg(row + p0 + m + 3);
      }
      key[m] = mass_key(v.x);
      key[m + 1] = mass_key(v.y);
      key[m + 2] = mass_key(v.z);
      key[m + 3] = mass_key(v.w);
    }
  };
  auto for_rounds = [&](auto&& f) {
    if (once) {
      f(lo);
    } else {
      for (int base = 0; base < s1; base += round) {
        load(base + lo);
        f(base + lo);
      }
    }
  };
  if (once) load(lo);

  uint32_t prefix = 0, pmask = 0, rem = (uint32_t)k;
  for (int i = tid; i < 3 * 2048; i += kSelThreads) (&hist[0][0])[i] = 0u;
  __syncthreads();
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, nb = pass == 2 ? 1024 : 2048;   // bits [21,32), [10,21), [0,10)
    const uint32_t dmask = (uint32_t)nb - 1u;
    uint32_t* h = hist[pass];
    for_rounds([&](int) {
#pragma unroll
      for (int m = 0; m < kPer; ++m)
        if (((in >> m) & 1u) && (key[m] & pmask) == prefix) atomicAdd(&h[(key[m] >> shift) & dmask], 1u);
    });
    if (C > 1) cluster_sync(); else __syncthreads();
    // digits in descending order, two per thread: where does the running count reach rem?
    const int d_hi = nb - 1 - 2 * tid, d_lo = nb - 2 - 2 * tid;
    uint32_t c_hi = 0, c_lo = 0;
    if (d_lo >= 0) {
      if (C == 1) {
        c_hi = h[d_hi];
        c_lo = h[d_lo];
      } else {
        uint32_t v_hi[kSelMaxCluster], v_lo[kSelMaxCluster];   // all remote loads first, then the sums
#pragma unroll
        for (uint32_t r = 0; r < kSelMaxCluster; ++r) {
          v_hi[r] = r < C ? ld_cluster_u32(mapa(smem_u32(&h[d_hi]), r)) : 0u;
          v_lo[r] = r < C ? ld_cluster_u32(mapa(smem_u32(&h[d_lo]), r)) : 0u;
        }
#pragma unroll
        for (uint32_t r = 0; r < kSelMaxCluster; ++r) {
          c_hi += v_hi[r];
          c_lo += v_lo[r];
        }
      }
    }
    uint32_t tot;
    const uint32_t above = scan_excl(c_hi + c_lo, hsum[pass], &tot);
    uint32_t* found = pick[pass];   // digit, entries above it, entries of it
    if (above < rem && rem <= above + c_hi) {
      found[0] = (uint32_t)d_hi;
      found[1] = above;
      found[2] = c_hi;
    } else if (above + c_hi < rem && rem <= above + c_hi + c_lo) {
      found[0] = (uint32_t)d_lo;
      found[1] = above + c_hi;
      found[2] = c_lo;
    }
    __syncthreads();
    rem -= found[1];
    prefix |= found[0] << shift;
    pmask |= dmask << shift;
    if (rem == found[2]) break;   // all of them stay: no lower digit decides anything
  }
  const uint32_t T = prefix;

  // Positions above T, and the first `rem` equal to T, in order. A round's CTAs follow one another:
  // each CTA's counts go to the higher ranks, the round's sum to the next round.
  uint32_t run_gt = 0, run_tie = 0, turn = 0;   // kept before this round, its number
  for_rounds([&](int p0) {
    uint32_t gt = 0, tie = 0;
#pragma unroll
    for (int m = 0; m < kPer; ++m) {
      if ((in >> m) & 1u) {
        gt += key[m] > T ? 1u : 0u;
        tie += key[m] == T ? 1u : 0u;
      }
    }
    uint64_t tot;
    const uint64_t ex = scan_excl(((uint64_t)gt << 32) | tie, wsum[turn & 1], &tot);
    ++turn;
    uint32_t g_before = run_gt + (uint32_t)(ex >> 32), t_before = run_tie + (uint32_t)ex;
    if (C == 1) {
      run_gt += (uint32_t)(tot >> 32);
      run_tie += (uint32_t)tot;
    } else {
      if (tid == 0) {
        slice[0] = (uint32_t)(tot >> 32);
        slice[1] = (uint32_t)tot;
      }
      cluster_sync();
      uint32_t v_gt[kSelMaxCluster], v_tie[kSelMaxCluster];
#pragma unroll
      for (uint32_t r = 0; r < kSelMaxCluster; ++r) {
        v_gt[r] = r < C ? ld_cluster_u32(mapa(smem_u32(&slice[0]), r)) : 0u;
        v_tie[r] = r < C ? ld_cluster_u32(mapa(smem_u32(&slice[1]), r)) : 0u;
      }
#pragma unroll
      for (uint32_t r = 0; r < kSelMaxCluster; ++r) {
        run_gt += v_gt[r];
        run_tie += v_tie[r];
        g_before += r < rank ? v_gt[r] : 0u;
        t_before += r < rank ? v_tie[r] : 0u;
      }
      cluster_sync();   // the counts are read before the next round, or before a CTA leaves
    }
#pragma unroll
    for (int m = 0; m < kPer; ++m) {
      if (!((in >> m) & 1u)) continue;
      if (key[m] > T) {
        out[s0 + g_before + min(t_before, rem)] = p0 + m;
        ++g_before;
      } else if (key[m] == T) {
        if (t_before < rem) out[s0 + g_before + t_before] = p0 + m;
        ++t_before;
      }
    }
  });
}

// ------------------------------------------------------------------------------ compact
constexpr int kCpThreads = 128;
constexpr int kCpRows = 8;                               // list entries per warp
constexpr int kCpSpan = kCpRows * (kCpThreads / 32);     // ... and per CTA
constexpr int kCpMaxSmem = 229376;

struct CompactArgs {
  int bs, num_blocks, max_blocks, dst_blocks, list_stride, mass_stride, mass_out_stride, B;
  uint8_t* cache;              // rows of row_bytes
  uint8_t* k_rope;             // E4M3: rows of kr_bytes, else null
  float* kv_scale;             // E4M3 only
  int row_bytes, kr_bytes;
  const int32_t* block_table;
  const int32_t* dst_table;
  const int32_t* indices;
  const int32_t* counts;
  const float* mass;           // null: no masses
  float* mass_out;
  int* status;
};

// (Plain loads here: the kernel may start while the one before it still writes, see the launch.)
// Lane i < 8 looks list entry j0 + i of sequence b up: its cache rows (dst < 0: none, or not to be
// copied). The entry's scale and mass move at once.
__device__ __forceinline__ void lookup(const CompactArgs& a, int b, int j0, int count, int& src, int& dst) {
  const int lane = threadIdx.x & 31, j = j0 + lane;
  src = 0;
  dst = -1;
  if (lane >= kCpRows) return;
  float m = 0.f;
  if (j < count) {
    const int t = a.indices[(size_t)b * a.list_stride + j];
    const int db = a.dst_table[(size_t)b * a.dst_blocks + j / a.bs];
    const bool ok_t = t >= 0 && t < a.max_blocks * a.bs;
    const int sb = ok_t ? a.block_table[(size_t)b * a.max_blocks + t / a.bs] : -1;
    const bool ok = sb >= 0 && sb < a.num_blocks && db >= 0 && db < a.num_blocks;
    if (ok) {
      src = sb * a.bs + t % a.bs;
      dst = db * a.bs + j % a.bs;
      if (a.kv_scale) a.kv_scale[dst] = a.kv_scale[src];
    } else {
      set_status(a.status, MLA_ERR_BAD_BLOCK_ID);
    }
    m = ok && a.mass && t < a.mass_stride ? a.mass[(size_t)b * a.mass_stride + t] : __uint_as_float(0x7FC00000u);
  }
  if (a.mass && j < a.mass_out_stride) a.mass_out[(size_t)b * a.mass_out_stride + j] = m;
}

__device__ __forceinline__ int list_count(const CompactArgs& a, int b) {
  int count = a.counts[b];
  if (count < 0 || count > a.list_stride) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, MLA_ERR_BAD_SEQ_LEN);
    count = min(max(count, 0), a.list_stride);
  }
  return count;
}

// Rows of whole 16-byte pieces, up to 7 KB: each of the warp's 8 lanes sends its row through shared
// memory with one bulk copy in and one out.
__global__ void __launch_bounds__(kCpThreads) cache_compact_bulk_kernel(const CompactArgs a, const uint64_t timeout_ns) {
  extern __shared__ __align__(128) uint8_t rows[];   // [kCpSpan][row_bytes + kr_bytes]
  __shared__ uint64_t bar[kCpThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t mine = smem_u32(&bar[warp]);
  if (lane == 0) {
    mbar_init(mine, 1);
    fence_mbarrier_init_cluster();
    fence_proxy_async_smem();
  }
  __syncwarp();
  const uint32_t kr = a.k_rope ? (uint32_t)a.kr_bytes : 0u, bytes = (uint32_t)a.row_bytes + kr;
  const uint32_t buf = smem_u32(rows) + (uint32_t)(warp * kCpRows + min(lane, kCpRows - 1)) * bytes;
  const int j0 = blockIdx.x * kCpSpan + warp * kCpRows;
  uint32_t phase = 0;
  int abort = 0;
  wait_for_grid_before();
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const int count = list_count(a, b);
    int src, dst;
    lookup(a, b, j0, count, src, dst);
    const unsigned go = __ballot_sync(0xffffffffu, dst >= 0);
    if (!go) continue;
    if (lane == 0) mbar_arrive_expect_tx(mine, (uint32_t)__popc(go) * bytes);
    __syncwarp();
    if (dst >= 0) {
      bulk_load(buf, a.cache + (size_t)src * a.row_bytes, a.row_bytes, mine);
      if (kr) bulk_load(buf + a.row_bytes, a.k_rope + (size_t)src * kr, kr, mine);
    }
    const bool ok = __all_sync(0xffffffffu, mbar_wait<false>(mine, phase, &abort, timeout_ns));
    if (!ok) {   // (copies in flight still write this buffer: wait for them without the short limit)
      if (lane == 0) set_status(a.status, MLA_ERR_TIMEOUT);
      int dummy = 0;
      mbar_wait<false>(mine, phase, &dummy, kDrainTimeoutNs);
      return;
    }
    phase ^= 1;
    if (dst >= 0) {
      bulk_store(a.cache + (size_t)dst * a.row_bytes, buf, a.row_bytes);
      if (kr) bulk_store(a.k_rope + (size_t)dst * kr, buf + a.row_bytes, kr);
      bulk_commit_group();
      bulk_wait_group_read<0>();   // the buffer is read before it is filled again, or the CTA leaves
    }
    __syncwarp();
  }
}

// Any rows: V-sized pieces (V divides both planes' rows and their bases' alignment) through registers,
// eight loads in flight per lane.
template <typename V>
__device__ __forceinline__ void copy_rows(uint8_t* base, int row_bytes, const int* src, const int* dst) {
  const int per = row_bytes / (int)sizeof(V), lane = threadIdx.x & 31;
#pragma unroll 1
  for (int i = lane; i < per; i += 32) {
    V v[kCpRows];
#pragma unroll
    for (int r = 0; r < kCpRows; ++r)
      if (dst[r] >= 0) v[r] = reinterpret_cast<const V*>(base + (size_t)src[r] * row_bytes)[i];
#pragma unroll
    for (int r = 0; r < kCpRows; ++r)
      if (dst[r] >= 0) reinterpret_cast<V*>(base + (size_t)dst[r] * row_bytes)[i] = v[r];
  }
}

template <typename V>
__global__ void __launch_bounds__(kCpThreads) cache_compact_kernel(const CompactArgs a) {
  const int j0 = blockIdx.x * kCpSpan + (threadIdx.x >> 5) * kCpRows;
  wait_for_grid_before();
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const int count = list_count(a, b);
    int my_src, my_dst;
    lookup(a, b, j0, count, my_src, my_dst);
    if (j0 >= count) continue;
    int src[kCpRows], dst[kCpRows];
#pragma unroll
    for (int r = 0; r < kCpRows; ++r) {
      src[r] = __shfl_sync(0xffffffffu, my_src, r);
      dst[r] = __shfl_sync(0xffffffffu, my_dst, r);
    }
    copy_rows<V>(a.cache, a.row_bytes, src, dst);
    if (a.k_rope) copy_rows<V>(a.k_rope, a.kr_bytes, src, dst);
  }
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }

}  // namespace
}  // namespace mla

extern "C" {

mla_status_t mla_evict_select(const mla_evict_params_t* p, const float* mass, const int32_t* seq_lens,
                              int32_t* indices, int32_t* counts, void* stream) {
  using namespace mla;
  if (!p || p->batch < 0 || p->max_seq_len < 0 || p->budget < 1 || p->sinks < 0 || p->recent < 0 ||
      (int64_t)p->sinks + p->recent > p->budget || p->reserved != 0)
    return MLA_ERR_INVALID_ARG;
  // (32-bit counters step over the rows of mass and indices)
  if (p->max_seq_len > (1 << 30) || p->budget > (1 << 30) || p->batch > (1 << 27)) return MLA_ERR_UNSUPPORTED;
  if (p->batch == 0) return MLA_OK;
  if (!mass || !seq_lens || !indices || !counts) return MLA_ERR_INVALID_ARG;
  const void* p4[] = {mass, seq_lens, indices, counts};
  for (const void* q : p4)
    if (!aligned(q, 4)) return MLA_ERR_ALIGNMENT;
  int* status = current_status_word();
  if (!status) return MLA_ERR_CUDA;
  const SelectArgs a{p->batch, p->max_seq_len, p->budget, p->sinks, p->recent, mass, seq_lens, indices, counts, status};
  int C = 1;
  while (C < kSelMaxCluster && C * kSelThreads * kSelPer < p->max_seq_len) C *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(p->batch * C));
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)C;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto kernel = p->max_seq_len <= kSelThreads * 4   ? evict_select_kernel<4>
                : p->max_seq_len <= kSelThreads * 8 ? evict_select_kernel<8>
                                                    : evict_select_kernel<kSelPer>;
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

mla_status_t mla_cache_compact(const mla_compact_params_t* p, void* kv_cache, void* k_rope_cache, float* kv_scale,
                               const int32_t* block_table, const int32_t* dst_block_table, const int32_t* indices,
                               const int32_t* counts, const float* mass, float* mass_out, void* stream) {
  using namespace mla;
  if (!p || p->batch < 0 || p->kv_rank < 1 || p->rope_dim < 0 || p->block_size < 1 || p->num_blocks < 0 ||
      p->max_blocks_per_seq < 1 || p->dst_max_blocks < 1 || p->list_stride < 1 || p->reserved != 0 ||
      (p->cache_dtype != MLA_DTYPE_F32 && p->cache_dtype != MLA_DTYPE_BF16 && p->cache_dtype != MLA_DTYPE_E4M3))
    return MLA_ERR_INVALID_ARG;
  if (p->batch > 0 && p->num_blocks < 1) return MLA_ERR_INVALID_ARG;
  if ((int64_t)p->dst_max_blocks * p->block_size < p->list_stride) return MLA_ERR_INVALID_ARG;
  if ((mass == nullptr) != (mass_out == nullptr)) return MLA_ERR_INVALID_ARG;
  if (mass && (p->mass_stride < 1 || p->mass_out_stride < p->list_stride)) return MLA_ERR_INVALID_ARG;
  if ((int64_t)p->max_blocks_per_seq * p->block_size > (1ll << 30) || (int64_t)p->kv_rank + p->rope_dim > (1 << 20) ||
      (int64_t)p->num_blocks * p->block_size > (1ll << 31) - 1 || p->list_stride > (1 << 30) ||
      (mass && (p->mass_stride > (1 << 30) || p->mass_out_stride > (1 << 30))))
    return MLA_ERR_UNSUPPORTED;
  if (p->batch == 0) return MLA_OK;
  if (!kv_cache || !block_table || !dst_block_table || !indices || !counts) return MLA_ERR_INVALID_ARG;
  const bool fp8 = p->cache_dtype == MLA_DTYPE_E4M3;
  if (fp8 ? (!kv_scale || (p->rope_dim > 0 && !k_rope_cache)) : (k_rope_cache || kv_scale)) return MLA_ERR_INVALID_ARG;
  if (block_table == dst_block_table) return MLA_ERR_INVALID_ARG;   // the destination blocks must be free
  // (a weight moves while others are read: in place, one block's writes would meet another's reads)
  if (mass && overlap(mass, 4ull * p->batch * p->mass_stride, mass_out, 4ull * p->batch * p->mass_out_stride))
    return MLA_ERR_INVALID_ARG;
  const void* p4[] = {block_table, dst_block_table, indices, counts, mass, mass_out, kv_scale};
  for (const void* q : p4)
    if (q && !aligned(q, 4)) return MLA_ERR_ALIGNMENT;
  if (!aligned(kv_cache, fp8 ? 1 : p->cache_dtype == MLA_DTYPE_BF16 ? 2 : 4) || (k_rope_cache && !aligned(k_rope_cache, 2)))
    return MLA_ERR_ALIGNMENT;
  int* status = current_status_word();
  if (!status) return MLA_ERR_CUDA;
  CompactArgs a{};
  a.bs = p->block_size;
  a.num_blocks = p->num_blocks;
  a.max_blocks = p->max_blocks_per_seq;
  a.dst_blocks = p->dst_max_blocks;
  a.list_stride = p->list_stride;
  a.mass_stride = p->mass_stride;
  a.mass_out_stride = p->mass_out_stride;
  a.B = p->batch;
  a.cache = (uint8_t*)kv_cache;
  a.k_rope = p->rope_dim > 0 ? (uint8_t*)k_rope_cache : nullptr;
  a.kv_scale = kv_scale;
  a.row_bytes = fp8 ? p->kv_rank : (p->kv_rank + p->rope_dim) * (p->cache_dtype == MLA_DTYPE_BF16 ? 2 : 4);
  a.kr_bytes = 2 * p->rope_dim;
  a.block_table = block_table;
  a.dst_table = dst_block_table;
  a.indices = indices;
  a.counts = counts;
  a.mass = mass;
  a.mass_out = mass_out;
  a.status = status;
  auto fits = [&](int u) {
    return a.row_bytes % u == 0 && aligned(a.cache, u) && (!a.k_rope || (a.kr_bytes % u == 0 && aligned(a.k_rope, u)));
  };
  const int span = mass ? p->mass_out_stride : p->list_stride;
  const dim3 grid((unsigned)((span + kCpSpan - 1) / kCpSpan), (unsigned)std::min(p->batch, 65535));
  cudaStream_t s = (cudaStream_t)stream;
  const int row_smem = kCpSpan * (a.row_bytes + (a.k_rope ? a.kr_bytes : 0));
  // A dependent of the kernel before it: behind a selection its blocks are in place when the lists are (both
  // calls, 64 sequences: 58.4 us behind a write-back of the L2, 56.4 like this).
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kCpThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t err = cudaSuccess;
  if (fits(16) && row_smem <= kCpMaxSmem) {
    static std::once_flag once[64];
    int dev = 0;
    cudaGetDevice(&dev);
    std::call_once(once[dev & 63], [&] {
      err = cudaFuncSetAttribute(cache_compact_bulk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCpMaxSmem);
    });
    if (err != cudaSuccess) return MLA_ERR_CUDA;
    cfg.dynamicSmemBytes = row_smem;
    err = cudaLaunchKernelEx(&cfg, cache_compact_bulk_kernel, a, wait_timeout_ns());
  } else if (fits(16)) {
    err = cudaLaunchKernelEx(&cfg, cache_compact_kernel<uint4>, a);
  } else if (fits(4)) {
    err = cudaLaunchKernelEx(&cfg, cache_compact_kernel<uint32_t>, a);
  } else {
    err = cudaLaunchKernelEx(&cfg, cache_compact_kernel<uint8_t>, a);
  }
  return err == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // extern "C"
