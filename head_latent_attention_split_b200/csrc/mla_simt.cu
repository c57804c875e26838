// CUDA-core kernels: the fp32 SIMT decode (any latent width, any block size, every
// storage type), the log-sum-exp combine of split partials, and the plan probe.
//
// SIMT decode: CTA (worker w, row block) with one warp per query row (s, h) of the
// sequence being processed. The worker's cache blocks are streamed through shared
// memory in chunks of tokens decoded to fp32 (bf16 / e4m3 * scale / f32); every warp
// scores the chunk against its row's absorbed query with an fp32 online softmax in
// base 2 (score * scale * log2 e) and accumulates the latent rows as values.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "mla_device.cuh"
#include "ptx_sm100.cuh"

namespace mla {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kChunkFloats = 12288;   // 48 KB of staged tokens

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void store_out(void* out, int dtype, size_t i, float v) {
  if (dtype == kF32) {
    ((float*)out)[i] = v;
  } else {
    // round to nearest even bf16 (finite inputs; NaN stays NaN)
    uint32_t u = __float_as_uint(v);
    uint16_t h;
    if ((u & 0x7FFFFFFFu) > 0x7F800000u)
      h = 0x7FC0;
    else
      h = (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
    ((uint16_t*)out)[i] = h;
  }
}

// kQV, kAV: per-lane query and accumulator registers (32 kQV >= r + d_r, 32 kAV >= r). Four tokens'
// dot products and their shuffles are under way together; the softmax then takes them one by one.
template <bool kWindow, int kQV, int kAV>
__global__ void __launch_bounds__(kThreads) simt_decode_kernel(const DecodeArgs a, int chunk) {
  extern __shared__ float tok[];   // [chunk][D]
  __shared__ WorkerPlan s_plan;
  const int D = a.r + a.d_r;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int w = blockIdx.x;
  const int row = blockIdx.y * kWarps + warp;
  const bool row_ok = row < a.rows;
  const int s = row_ok ? row / a.H : 0;
  const int cap = a.len_cap;
  const auto tiles = TilesOf<kWindow>::make(a);   // windowed: only the blocks that some row sees
  if constexpr (kWindow) ptx::launch_dependents();   // the combine

  if (warp == 0) {
    WorkerPlan p = warp_plan(a.seq_lens, a.B, tiles, cap, a.W, w, a.status);
    if (lane == 0) s_plan = p;
  }
  __syncthreads();
  const WorkerPlan plan = s_plan;

  SegmentIterT<typename TilesOf<kWindow>::type> it(plan, a.seq_lens, a.B, tiles, cap, w, a.status);
  Segment sg;
  while (it.next(sg)) {
    const int b = sg.b;
    if (sg.split == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
      a.meta[2 * b] = sg.first_worker;
      a.meta[2 * b + 1] = sg.splits;
    }
    // absorbed query of this row, lane-strided
    float q[kQV];
    const size_t qrow = (size_t)b * a.rows + row;
#pragma unroll
    for (int i = 0; i < kQV; ++i) {
      const int k = lane + 32 * i;
      float v = 0.f;
      if (row_ok && k < a.r) v = load_q(a.q_lat, a.q_dtype, qrow * a.r + k);
      else if (row_ok && k < D) v = load_q(a.q_rope, a.q_dtype, qrow * a.d_r + (k - a.r));
      q[i] = v;
    }
    float acc[kAV];
#pragma unroll
    for (int i = 0; i < kAV; ++i) acc[i] = 0.f;
    float m = -INFINITY, l = 0.f;

    // the segment's tokens are runs of consecutive positions: one, or two around the gap
    // between the sink blocks and the window's
    const int n_row = a.causal ? sg.Lc - a.Sq + 1 + s : sg.Lc;   // tokens this row may see
    const int n_runs = kWindow ? 2 : 1;
    for (int run = 0; run < n_runs; ++run) {
      int t_begin = sg.tile_begin * a.bs, t_end = min(sg.tile_end * a.bs, sg.Lc);
      int lo = 0, sink = 0;   // the row sees tokens t < n_row with t >= lo or t < sink
      if constexpr (kWindow) {
        const int st = tiles.sink_tiles(sg.Lc), gap = tiles.gap(sg.Lc);
        const int i0 = run == 0 ? sg.tile_begin : max(sg.tile_begin, st);
        const int i1 = run == 0 ? min(sg.tile_end, st) : sg.tile_end;
        t_begin = (i0 + (run ? gap : 0)) * a.bs;
        t_end = min((i1 + (run ? gap : 0)) * a.bs, sg.Lc);
        lo = n_row - a.window;
        sink = a.sinks;
      }
      const int hi = min(t_end, n_row);
      for (int c0 = t_begin; c0 < t_end; c0 += chunk) {
        const int cn = min(chunk, t_end - c0);
        __syncthreads();
        // the chunk's values as one flat list over the block: the loads do not wait for one another
#pragma unroll 4
        for (int i = threadIdx.x; i < cn * D; i += kThreads) {
          const int j = i / D, k = i - j * D, t = c0 + j;
          const int blk = checked_block(a.block_table, a.max_blocks, b, t / a.bs, a.num_blocks, a.status);
          const size_t slot = (size_t)blk * a.bs + (t % a.bs);
          float v;
          if (a.cache_dtype == kE4M3) {
            if (k < a.r)
              v = e4m3_to_float(__ldg((const uint8_t*)a.cache + slot * a.r + k)) * __ldg(a.kv_scale + slot);
            else
              v = bf16_bits_to_float(__ldg(a.k_rope + slot * a.d_r + (k - a.r)));
          } else if (a.cache_dtype == kBF16) {
            v = bf16_bits_to_float(__ldg((const uint16_t*)a.cache + slot * D + k));
          } else {
            v = __ldg((const float*)a.cache + slot * D + k);
          }
          tok[i] = v;
        }
        __syncthreads();
        if (!row_ok) continue;
        const int jn = min(cn, hi - c0);
        constexpr int kT = 4;
        for (int j0 = 0; j0 < jn; j0 += kT) {
          float x[kT];
#pragma unroll
          for (int u = 0; u < kT; ++u) {
            const float* c = tok + min(j0 + u, jn - 1) * D;
            float d = 0.f;
#pragma unroll
            for (int i = 0; i < kQV; ++i) {
              const int k = lane + 32 * i;
              if (k < D) d = fmaf(q[i], c[k], d);
            }
            x[u] = d;
          }
#pragma unroll
          for (int u = 0; u < kT; ++u) x[u] = warp_sum(x[u]) * a.scale_log2;
#pragma unroll
          for (int u = 0; u < kT; ++u) {
            const int j = j0 + u;
            if (j >= jn || (kWindow && c0 + j < lo && c0 + j >= sink)) continue;   // not seen by this row
            const float* c = tok + j * D;
            const float m_new = fmaxf(m, x[u]);
            const float corr = exp2f(m - m_new);
            const float p = exp2f(x[u] - m_new);
            l = fmaf(l, corr, p);
#pragma unroll
            for (int i = 0; i < kAV; ++i) {
              const int k = lane + 32 * i;
              if (k < a.r) acc[i] = fmaf(acc[i], corr, p * c[k]);
            }
            m = m_new;
          }
        }
      }
    }
    const bool poisoned = segment_poisoned(a, tiles, b, sg.tile_begin, sg.tile_end);
    if (!row_ok) continue;
    const float qnan = __uint_as_float(0x7FC00000u);
    const float inv = poisoned ? qnan : l > 0.f ? 1.f / l : 0.f;
    const float lse_v = poisoned ? qnan : l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
    if (sg.splits == 1) {
#pragma unroll
      for (int i = 0; i < kAV; ++i) {
        const int k = lane + 32 * i;
        if (k < a.r) store_out(a.out, a.out_dtype, qrow * a.r + k, acc[i] * inv);
      }
      if (lane == 0) a.lse[qrow] = lse_v;
    } else {
      const size_t prow = (size_t)(w + b) * a.rows + row;
#pragma unroll
      for (int i = 0; i < kAV; ++i) {
        const int k = lane + 32 * i;
        if (k < a.r) a.o_part[prow * a.r + k] = acc[i] * inv;
      }
      if (lane == 0) a.lse_part[prow] = lse_v;
    }
  }
}

// One row's output and log-sum-exp from its `splits` partials (not 1), by one warp; none: zeros, or NaN behind a
// length that is out of range. kMany: many rows per warp slot, where resident warps hide the latencies; else the
// first partials are requested before their weights are known.
template <bool kMany>
__device__ __forceinline__ void combine_row(const DecodeArgs& a, int b, int row, int first, int splits, bool bad) {
  const int lane = threadIdx.x & 31;
  const size_t orow = (size_t)b * a.rows + row;
  const float qnan = __uint_as_float(0x7FC00000u);
  if (splits == 0) {
    for (int k = lane; k < a.r; k += 32) store_out(a.out, a.out_dtype, orow * a.r + k, bad ? qnan : 0.f);
    if (lane == 0) a.lse[orow] = bad ? qnan : -INFINITY;
    return;
  }
  const size_t slot0 = (size_t)first + b;
  const bool vec = a.r % 4 == 0;
  // the first two splits' pieces of the first 512 channels (see below), requested at once
  constexpr int kEarly = kMany ? 0 : 2;
  float4 early[2][4];
#pragma unroll
  for (int i = 0; i < kEarly; ++i) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = 4 * lane + 128 * u;
      early[i][u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (vec && k < a.r) early[i][u] = *reinterpret_cast<const float4*>(a.o_part + ((slot0 + i) * a.rows + row) * a.r + k);
    }
  }
  float M = -INFINITY, mine = -INFINITY;   // mine: the log-sum-exp of split `lane`
  bool has_nan = false;
  for (int i = lane; i < splits; i += 32) {
    const float v = a.lse_part[(slot0 + i) * a.rows + row];
    if (i == lane) mine = v;
    has_nan |= v != v;
    M = fmaxf(M, v);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (__any_sync(0xffffffffu, has_nan)) {
    for (int k = lane; k < a.r; k += 32) store_out(a.out, a.out_dtype, orow * a.r + k, qnan);
    if (lane == 0) a.lse[orow] = qnan;
    return;
  }
  if (M == -INFINITY) {
    for (int k = lane; k < a.r; k += 32) store_out(a.out, a.out_dtype, orow * a.r + k, 0.f);
    if (lane == 0) a.lse[orow] = -INFINITY;
    return;
  }
  float Z = 0.f;
  for (int i = lane; i < splits; i += 32) Z += expf((i == lane ? mine : a.lse_part[(slot0 + i) * a.rows + row]) - M);
  Z = warp_sum(Z);
  const float lse_v = M + logf(Z);
  if (vec) {
    // 512 channels per pass, 16 per lane as four float4 pieces; each split's pieces are
    // independent loads, so a split costs one memory latency, not one per piece. The split
    // weights come from lane i (splits <= 32) by shuffle; the output goes out 4 channels per store.
    const float wl = lane < splits ? expf(mine - lse_v) : 0.f;
    // 4 output channels per store when the output allows it (the SIMT path takes 4-byte
    // aligned outputs)
    const bool vec_out = ((uintptr_t)a.out % (a.out_dtype == kF32 ? 16u : 8u)) == 0;
    for (int k0 = 0; k0 < a.r; k0 += 512) {
      float4 o[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      auto add = [&](float wgt, const float4* v) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          o[u].x = fmaf(wgt, v[u].x, o[u].x);
          o[u].y = fmaf(wgt, v[u].y, o[u].y);
          o[u].z = fmaf(wgt, v[u].z, o[u].z);
          o[u].w = fmaf(wgt, v[u].w, o[u].w);
        }
      };
      int i0 = 0;
      if (k0 == 0) {   // (splits >= 2)
#pragma unroll
        for (int i = 0; i < kEarly; ++i) {
          const float wgt = __shfl_sync(0xffffffffu, wl, i);
          if (wgt != 0.f) add(wgt, early[i]);
        }
        i0 = kEarly;
      }
      // splits whose pieces are on their way together, added in order (1 sequence of 65 tiles in 17 parts: 36.0 us
      // with 2, 37.0 with 3, 38.2 with 4, whose registers spill)
      constexpr int kG = kMany ? 1 : 2;
#pragma unroll 1
      for (int i = i0; i < splits; i += kG) {
        float4 v[kG][4];
        float late[kG];       // log-sum-exps behind the 32 that the lanes hold
#pragma unroll
        for (int j = 0; j < kG; ++j) {
          const size_t prow = (slot0 + i + j) * a.rows + row;
          const float* src = a.o_part + prow * a.r;
          late[j] = i + j >= 32 && i + j < splits ? a.lse_part[prow] : 0.f;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int k = k0 + 4 * lane + 128 * u;
            v[j][u] = i + j < splits && k < a.r ? *reinterpret_cast<const float4*>(src + k) : make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
#pragma unroll
        for (int j = 0; j < kG; ++j) {
          const float held = __shfl_sync(0xffffffffu, wl, (i + j) & 31);
          const float wgt = i + j >= splits ? 0.f : i + j < 32 ? held : expf(late[j] - lse_v);
          if (wgt != 0.f) add(wgt, v[j]);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = k0 + 4 * lane + 128 * u;
        if (k < a.r && !vec_out) {
          const size_t e = orow * a.r + k;
          store_out(a.out, a.out_dtype, e, o[u].x);
          store_out(a.out, a.out_dtype, e + 1, o[u].y);
          store_out(a.out, a.out_dtype, e + 2, o[u].z);
          store_out(a.out, a.out_dtype, e + 3, o[u].w);
        } else if (k < a.r) {
          const size_t e = orow * a.r + k;
          if (a.out_dtype == kF32) {
            *reinterpret_cast<float4*>((float*)a.out + e) = o[u];
          } else {
            uint32_t lo, hi;   // round to nearest even; NaN stays NaN
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(o[u].y), "f"(o[u].x));
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(o[u].w), "f"(o[u].z));
            *reinterpret_cast<uint2*>((uint16_t*)a.out + e) = make_uint2(lo, hi);
          }
        }
      }
    }
  } else {
    for (int k0 = 0; k0 < a.r; k0 += 32 * 4) {
      float o[4] = {0.f, 0.f, 0.f, 0.f};
      for (int i = 0; i < splits; ++i) {
        const size_t prow = (slot0 + i) * a.rows + row;
        const float wgt = expf(a.lse_part[prow] - lse_v);
        if (wgt == 0.f) continue;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int k = k0 + lane + 32 * u;
          if (k < a.r) o[u] = fmaf(wgt, a.o_part[prow * a.r + k], o[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = k0 + lane + 32 * u;
        if (k < a.r) store_out(a.out, a.out_dtype, orow * a.r + k, o[u]);
      }
    }
  }
  if (lane == 0) a.lse[orow] = lse_v;
}

// One warp per (b, row): merge the partials of split sequences, fill empty ones. The split of
// each sequence is recomputed here from seq_lens with the plan's formula (nothing read from the
// workspace is trusted for indexing). Rows of a sequence with a seq_len out of range, and rows
// whose partials carry a NaN log-sum-exp (a decode wait timed out, or a bad block id), are
// written as NaN.
// A chain of latencies bounds it (a few MB of partials, in L2): lengths, log-sum-exps, partials. So the
// window decode launches it as a dependent of the decode kernel, with the lengths read and the
// split found while that kernel still runs, and the partials of the first splits are requested before
// their weights are known.
template <bool kWindow, bool kMany>
__global__ void __launch_bounds__(kThreads, kMany ? 4 : 2) combine_kernel(const DecodeArgs a) {
  __shared__ long long s_sum[kWarps][2];
  __shared__ int s_most[kWarps][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x;
  const int cap = a.len_cap;
  const auto tiles = TilesOf<kWindow>::make(a);
  // tiles before sequence b and in total, as the decode kernels' plan counts them
  long long before = 0, total = 0;
  int most = 0, hidden = 0;
  for (int i = threadIdx.x; i < a.B; i += kThreads) {
    const int L = __ldg(a.seq_lens + i), Lc = L < 0 ? 0 : (L > cap ? cap : L);
    const int n = tiles.count(Lc);
    total += n;
    most = max(most, n);
    hidden = max(hidden, tiles.gap(Lc));
    if (i < b) before += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  hidden = __reduce_max_sync(0xffffffffu, hidden);
  if (lane == 0) {
    s_sum[warp][0] = before;
    s_sum[warp][1] = total;
    s_most[warp][0] = most;
    s_most[warp][1] = hidden;
  }
  __syncthreads();
  before = total = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    before += s_sum[i][0];
    total += s_sum[i][1];
    most = max(most, s_most[i][0]);
    hidden = max(hidden, s_most[i][1]);
  }
  const int raw = __ldg(a.seq_lens + b);
  const float qnan = __uint_as_float(0x7FC00000u);
  const long long n = raw < 0 || raw > cap ? 0 : tiles.count(raw);
  int first = 0, splits = 0;
  int cut = 0;
  if constexpr (kWindow) cut = tiles.cut(total, most, hidden, a.B, a.W);
  if (n > 0 && cut) {
    const int parts = max(-cut, 1);
    first = b * parts;
    splits = (int)min((long long)parts, n);
  } else if (n > 0) {
    const int Wa = (total < a.W) ? (int)total : a.W;
    first = worker_of_tile(before, total, Wa);
    splits = worker_of_tile(before + n - 1, total, Wa) - first + 1;
  }
  if constexpr (kWindow) ptx::wait_for_grid_before();   // every thread, so that this grid ends after the decode's
  if (splits == 1) return;                              // (the decode wrote the rows directly)
  for (int row = blockIdx.y * kWarps + warp; row < a.rows; row += gridDim.y * kWarps)
    combine_row<kMany>(a, b, row, first, splits, raw < 0 || raw > cap);
}

__global__ void __launch_bounds__(32) plan_probe_kernel(const DecodeArgs a, int32_t* token_slot,
                                                         int32_t* token_worker) {
  const int w = blockIdx.x, lane = threadIdx.x;
  const int cap = a.len_cap;
  const WorkerPlan p = warp_plan(a.seq_lens, a.B, a.bs, cap, a.W, w, a.status);
  SegmentIter it(p, a.seq_lens, a.B, a.bs, cap, w, a.status);
  Segment sg;
  while (it.next(sg)) {
    if (sg.split == 0 && lane == 0) {
      a.meta[2 * sg.b] = sg.first_worker;
      a.meta[2 * sg.b + 1] = sg.splits;
    }
    const int t1 = min(sg.tile_end * a.bs, sg.Lc);
    for (int t = sg.tile_begin * a.bs + lane; t < t1; t += 32) {
      const int blk = checked_block(a.block_table, a.max_blocks, sg.b, t / a.bs, a.num_blocks, a.status);
      const size_t o = (size_t)sg.b * a.max_blocks * a.bs + t;
      token_slot[o] = blk * a.bs + t % a.bs;
      token_worker[o] = w;
    }
  }
}

}  // namespace

cudaError_t launch_simt_decode(const DecodeArgs& a, cudaStream_t s) {
  const int D = a.r + a.d_r;
  int chunk = kChunkFloats / D;
  if (chunk > 32) chunk = 32;
  if (chunk < 1) chunk = 1;
  dim3 grid(a.W, (a.rows + kWarps - 1) / kWarps);
  // the registers of the widest shapes, or of those up to 128 wide (a call on a tiny window of 24-wide rows:
  // 57 us with 40 + 32 registers and one token at a time; 20 us like this, which the host takes to launch it)
  constexpr int kWQ = kSimtMaxD / 32, kWA = kSimtMaxR / 32;
  auto kernel = D <= 128 ? (a.window > 0 ? simt_decode_kernel<true, 4, 4> : simt_decode_kernel<false, 4, 4>)
                         : (a.window > 0 ? simt_decode_kernel<true, kWQ, kWA> : simt_decode_kernel<false, kWQ, kWA>);
  kernel<<<grid, kThreads, sizeof(float) * chunk * D, s>>>(a, chunk);
  return cudaGetLastError();
}

cudaError_t launch_combine(const DecodeArgs& a, cudaStream_t s) {
  // Up to two blocks per SM with one per eight rows: latency decides, and the variant of 118 registers has the first
  // partials under way early. Beyond, resident warps do, with 61 registers. A step with the one and the other, us
  // (sequences x rows, from a cold L2; the rule's side first):
  //   up to two: window 16 x 32 39.3, 41.0; 1 x 128 of 65 tiles 43.0, 47.2; 8 x 128 51.2, 53.4; dense 18 x 128 80.3, 82.0;
  //   beyond: window 24 x 128 70.0, 72.2; 32 x 128 e4m3 83.5, 86.1; 96 ragged x 256 145.4, 151.6; dense 24 ragged x 128
  //   59.6, 61.6; 128 ragged x 256 159.7, 170.6; but window 30 ragged x 256 69.6, 68.2.
  // Beyond, a dense batch keeps a block per eight rows, since its sequences' splits differ (128 ragged x 256: 159.7,
  // 163.9 when four blocks per SM walk the rows; 64 x 128: 178.1, 176.1). The blocks of a window batch walk them:
  // there it is a draw (30 ragged x 256: 69.6, 71.6 with a block per eight rows; 96 ragged x 256 145.4 both; 40
  // ragged x 128 90.0, 86.0), and blocks of sequences that need no merge are fewer.
  int dev = 0, sms = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (err != cudaSuccess) return err;
  const int groups = (a.rows + kWarps - 1) / kWarps, batch = std::max(a.B, 1);
  const bool many = (int64_t)groups * batch > 2 * sms;
  const int walk = std::max(1, std::min(groups, (many ? 4 : 2) * sms / batch));
  const dim3 grid(a.B, many && a.window == 0 ? groups : walk);
  if (a.window > 0) {
    // a dependent of the decode kernel before it: its blocks may start while that kernel's last CTAs run
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return many ? cudaLaunchKernelEx(&cfg, combine_kernel<true, true>, a) : cudaLaunchKernelEx(&cfg, combine_kernel<true, false>, a);
  }
  if (many)
    combine_kernel<false, true><<<grid, kThreads, 0, s>>>(a);
  else
    combine_kernel<false, false><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_plan_probe(const DecodeArgs& a, int32_t* token_slot, int32_t* token_worker,
                              cudaStream_t s) {
  plan_probe_kernel<<<a.W, 32, 0, s>>>(a, token_slot, token_worker);
  return cudaGetLastError();
}

}  // namespace mla
