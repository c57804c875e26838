// Attention weight per cached token (mla_attention_mass in include/mla_decode.h):
//   mass[b, t] = mass_in[b, t] + sum over rows (s, h) that see t of exp(sigma_t(s, h) - lse[b, s, h]).
//
// mass_simt_kernel: fp32 CUDA cores, any width, block size and storage type. A CTA takes 32 tokens
// of one sequence, decoded to fp32 in shared memory; lane = token, a warp takes every eighth group
// of four query rows, so one token value serves four products. Bound by the fp32 products (and the
// shared-memory reads that feed them); it serves the shapes the tensor kernel does not take.
//
// mass_tc_kernel (r = 512, d_r = 64, 64-token blocks, bf16 or e4m3 cache): one pass over the cache on
// the tensor cores, persistent, one CTA per SM on a contiguous range of 128-token tiles. The TOKENS
// are the MMA's M = 128 and the query rows its N (up to 128), so a TMEM lane holds one token's
// scores of all rows and the thread that reads it sums exp2(score - lse) alone: no exchange
// between threads, one coalesced store. The query (9 chunks of 64 channels, 147 KB at 128 rows) stays
// in shared memory for a whole run of tiles, and what is left of shared memory is a ring of 16 KB
// cache chunks (two TMA boxes, one per block) in flight. More than 128 rows go in groups, over
// runs of four tiles at a time (150 * 4 * 147 KB: the second group's reads hit L2); a token's sum over
// the groups is added up by one thread, in order.
// With an e4m3 cache the codes are an operand as they are (kind::f8f6f4): the bf16 query is split into
// an e4m3 and an e5m2 term (8 = 4 + 4 significant bits, see split_f8), both multiplied into one accumulator,
// and the RoPE part has its own bf16 MMAs and accumulator since the token's scale does not apply to
// it. No conversion of cache data at all.
// Bound: memory. Per 128 tokens and SM 36 MMAs of N = 128 take about 2.9 k cycles and the
// exponentials about 1.1 k (16 per cycle), the tile's bytes at 1/148 of the HBM rate 6.4 k (bf16)
// or 3.6 k (e4m3). Measured at 128 heads: bf16, 64 sequences of 8192: 111 us (5.4 TB/s; up to 124 us in long
// runs under the power cap); e4m3, 48 sequences of up to 16384: 64 us (2.8 TB/s). What is missing is
// the ring: 80 KB in flight per SM beside the query, at about 2.2 us of latency under load, and with an
// e4m3 cache the start of each sequence's tiles behind its query. An L2 prefetch of the blocks ahead made it
// slower (117 to 122 us and more), other L2 promotion sizes changed nothing.
#include <cuda.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "mla_device.cuh"
#include "ptx_sm100.cuh"

namespace mla {
namespace {

using namespace ptx;

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

// ------------------------------------------------------------------------ tensor cores
constexpr int kR = 512, kDR = 64, kBS = 64;
constexpr int kTile = 128;                       // tokens per tile = MMA M: two cache blocks
constexpr uint32_t kBox = kBS * 128;             // 64 tokens x 128 bytes, 128-byte swizzle
constexpr uint32_t kSlot = 2 * kBox;             // one chunk of a tile
constexpr int kMaxSlots = 12;
constexpr int kQChunks = 9;                      // query: 9 x [N rows][128 bytes]
constexpr int kGroupRows = 128;                  // query rows per group (at most)
constexpr int kGroupRun = 4;                     // tiles per run when there are several groups
// warps 0-7 sums (0-3 the even tiles, 4-7 the odd ones) and, for an e4m3 cache, the query's split; 8 TMA, 9 MMA
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr int kTcThreads = 32 * 10;
constexpr uint32_t kCtlBytes = 2048;             // leaves 5 ring slots at 128 rows
constexpr uint32_t kSmemMax = 232448;

// What the producer tells the MMA warp about a tile, released by the tile's first chunk. The producer is
// ahead of it by the ring at most (12 chunks: two tiles and a part), so eight slots do.
constexpr int kTileFlags = 8;
enum : uint32_t { kFirst = 1, kLast = 2, kStop = 4 };   // tile of an item; no more tiles

struct MassCtl {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t q_full[kQChunks], q_empty[kQChunks];   // e4m3: [0] the split latent part, [8] the RoPE part
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  WorkerPlan plan;
  alignas(16) float nl2[kGroupRows];   // -lse * log2(e) of the group's rows; -inf for rows that are none
  alignas(16) float a2[kGroupRows];    // e4m3: the row's power of two * scale * log2(e)
  uint8_t late[kGroupRows];  // causal: query tokens between the group's first row and this one
  uint32_t flags[kTileFlags];
};
static_assert(sizeof(MassCtl) <= kCtlBytes, "control block");

// One query row (16 channels per lane, v = 8 bf16 pairs) as hi + lo terms of x * 2^-e (split_f8);
// returns the exponent field of 2^e.
__device__ __forceinline__ uint32_t split_row(const uint32_t* v, uint32_t* hi, uint32_t* lo) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, bf16x2_amax(v[i]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int e = split_exponent(m);
  const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
  for (int i = 0; i < 4; ++i) split_f8(v[2 * i], v[2 * i + 1], down, hi[i], lo[i]);
  return (uint32_t)(127 + e);
}

template <bool kFp8>
__global__ void __launch_bounds__(kTcThreads, 1)
    mass_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_qr,
                   const __grid_constant__ CUtensorMap tm_kv, const __grid_constant__ CUtensorMap tm_kr,
                   const MassArgs m, const int N, const int slots, const uint64_t timeout_ns, const uint64_t drain_ns) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const DecodeArgs& a = m.d;
  const uint32_t q_chunk = (uint32_t)N * 128;            // bytes of one query chunk
  const uint32_t sRing = smem_u32(smem), sQ = sRing + (uint32_t)slots * kSlot;
  uint8_t* gQ = smem + (uint32_t)slots * kSlot;
  MassCtl& ctl = *reinterpret_cast<MassCtl*>(gQ + kQChunks * q_chunk);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &ctl.abort;
  constexpr int kChunks = kFp8 ? 5 : 9;                  // cache chunks per tile, the last one RoPE
  constexpr uint32_t kTmemCols = kFp8 ? 512 : 256;       // two accumulator stages
  constexpr uint32_t kAccCols = kTmemCols / 2;
  constexpr float kLog2e = 1.4426950408889634f;
  const DenseTiles tiles(kTile);
  const int n_groups = (a.rows + kGroupRows - 1) / kGroupRows;

  if (warp == kTmaWarp) {
    const WorkerPlan p = warp_plan(a.seq_lens, a.B, tiles, a.len_cap, a.W, blockIdx.x, a.status);
    if (lane == 0) {
      ctl.plan = p;
      prefetch_tmap(&tm_q);
      prefetch_tmap(&tm_kv);
    }
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < slots; ++i) {
      mbar_init(smem_u32(&ctl.full[i]), 1);
      mbar_init(smem_u32(&ctl.empty[i]), 1);
    }
    for (int i = 0; i < kQChunks; ++i) {
      mbar_init(smem_u32(&ctl.q_full[i]), kFp8 && i == 0 ? 8 : 1);   // e4m3: one arrival per sum warp
      mbar_init(smem_u32(&ctl.q_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ctl.acc_full[i]), 1);
      mbar_init(smem_u32(&ctl.acc_empty[i]), 4);   // one arrival per sum warp of the tile
    }
    mbar_init(smem_u32(&ctl.drain), 1);
    ctl.abort = 0;
    fence_mbarrier_init_cluster();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&ctl.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;

  // The CTA's items in order, the same walk in every role: f(b, Lc, group, first tile, end tile) for
  // a run of tiles of one sequence and one group of rows. Sequences with a bad length have none.
  auto for_items = [&](auto&& f) {
    SegmentIterT<DenseTiles> it(ctl.plan, a.seq_lens, a.B, tiles, a.len_cap, blockIdx.x, a.status);
    Segment sg;
    bool ok = true;
    while (ok && it.next(sg)) {
      const int L = __ldg(a.seq_lens + sg.b);
      if (L < 0 || L > a.len_cap) continue;
      const int run = n_groups == 1 ? sg.tile_end - sg.tile_begin : kGroupRun;
      for (int t0 = sg.tile_begin; ok && t0 < sg.tile_end; t0 += run)
        for (int g = 0; ok && g < n_groups; ++g) ok = f(sg.b, sg.Lc, g, t0, min(t0 + run, sg.tile_end));
    }
    return ok;
  };

  if (warp == kTmaWarp) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      int slot = 0, issued = 0;
      uint32_t phase = 0, item = 0, u = 0, q_issued = 0;   // u: tiles; q_issued: query chunks loaded so far
      const bool ok = for_items([&](int b, int Lc, int g, int t0, int t1) {
        if constexpr (kFp8)   // the sum warps' reads of the item's query, a ring's time early (64.9 us without, 63.1)
          prefetch_l2((const uint16_t*)a.q_lat + ((size_t)b * a.rows + g * kGroupRows) * kR,
                      (uint32_t)min(a.rows - g * kGroupRows, kGroupRows) * kR * 2);
        const int32_t* bt = a.block_table + (size_t)b * a.max_blocks;
        const int blocks = tiles_of(Lc, kBS);
        int next[2] = {__ldg(bt + 2 * t0), 2 * t0 + 1 < blocks ? __ldg(bt + 2 * t0 + 1) : 0};
        for (int t = t0; t < t1; ++t) {
          int blk[2];
          const int nblk = min(blocks - 2 * t, 2);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            blk[h] = next[h];
            if (blk[h] < 0 || blk[h] >= a.num_blocks) blk[h] = a.num_blocks;   // past the cache: reads zeros
            const int ahead = 2 * (t + 1) + h;   // the next tile's ids, a tile's time early
            next[h] = t + 1 < t1 && ahead < blocks ? __ldg(bt + ahead) : 0;
          }
#pragma unroll 1
          for (int j = 0; j < kChunks; ++j) {
            const bool rope = j == kChunks - 1;
            if (t == t0 && (!kFp8 || rope)) {   // the item's query chunk (e4m3: the sum warps write the latent part)
              const int qj = rope ? kQChunks - 1 : j;
              if (!mbar_wait<false>(smem_u32(&ctl.q_empty[qj]), (item & 1) ^ 1, abort, timeout_ns)) return false;
              const uint32_t bar = smem_u32(&ctl.q_full[qj]);
              mbar_arrive_expect_tx(bar, q_chunk);
              tma_load_3d(sQ + qj * q_chunk, rope ? &tm_qr : &tm_q, bar, rope ? 0 : 64 * j, g * kGroupRows, b);
              ++q_issued;
            }
            if (!mbar_wait<false>(smem_u32(&ctl.empty[slot]), phase ^ 1, abort, timeout_ns)) return false;
            if (j == 0) ctl.flags[u++ % kTileFlags] = (t == t0 ? kFirst : 0u) | (t == t1 - 1 ? kLast : 0u);
            const uint32_t bar = smem_u32(&ctl.full[slot]);
            mbar_arrive_expect_tx(bar, nblk * kBox);
            for (int h = 0; h < nblk; ++h) {
              const uint32_t dst = sRing + slot * kSlot + h * kBox;
              if constexpr (kFp8) {
                if (rope)
                  tma_load_3d(dst, &tm_kr, bar, 0, 0, blk[h]);
                else
                  tma_load_3d(dst, &tm_kv, bar, 128 * j, 0, blk[h]);
              } else {
                tma_load_3d(dst, &tm_kv, bar, 64 * j, 0, blk[h]);
              }
            }
            ++issued;
            if (++slot == slots) {
              slot = 0;
              phase ^= 1;
            }
          }
        }
        ++item;
        return true;
      });
      // the end, in place of a tile's first chunk
      const bool stop = ok && mbar_wait<false>(smem_u32(&ctl.empty[slot]), phase ^ 1, abort, timeout_ns);
      if (stop) {
        ctl.flags[u % kTileFlags] = kStop;
        mbar_arrive(smem_u32(&ctl.full[slot]));
      }
      // every load issued lands before the CTA may exit (the one that was in the end's slot has)
      int dummy = 0;
      for (int i = max(0, issued - slots + (stop ? 1 : 0)); i < issued; ++i)
        mbar_wait<false>(smem_u32(&ctl.full[i % slots]), (i / slots) & 1, &dummy, drain_ns);
      if (!ok) {   // the query chunks of an unfinished item too
        constexpr uint32_t per = kFp8 ? 1 : kQChunks;
        for (uint32_t i = q_issued > per ? q_issued - per : 0; i < q_issued; ++i)
          mbar_wait<false>(smem_u32(&ctl.q_full[kFp8 ? kQChunks - 1 : i % per]), (i / per) & 1, &dummy, drain_ns);
        set_status(a.status, MLA_ERR_TIMEOUT);
      }
    }
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- MMA issuer (a converged warp)
    const bool leader = elect_one();
    const uint32_t idesc16 = idesc_bf16_f32(kTile, N, false), idesc8 = idesc_e4m3_f32(kTile, N),
                   idesc8lo = idesc_f8_f32(kTile, N, false, true);
    // operand descriptors of ring slot 0 and query chunk 0; a step of 32 bytes (K = 16 bf16 or 32 codes) adds 2
    const uint64_t ring_desc = smem_desc(sRing, 16, 1024, kSwizzle128B), q_desc = smem_desc(sQ, 16, 1024, kSwizzle128B);
    auto wait = [&](uint64_t& bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait<false>(smem_u32(&bar), parity, abort, timeout_ns));
    };
    int slot = 0;
    uint32_t phase = 0, item = 0, u = 0;
    bool ok;
    while ((ok = wait(ctl.full[slot], phase))) {   // the tile's first chunk, or the end
      const uint32_t flags = __shfl_sync(0xffffffffu, ctl.flags[u % kTileFlags], 0);
      if (flags & kStop) break;
      ok = wait(ctl.acc_empty[u & 1], ((u >> 1) & 1) ^ 1);
      const uint32_t d = tmem + (u & 1) * kAccCols;
#pragma unroll 1
      for (int j = 0; ok && j < kChunks; ++j) {
        const bool rope = j == kChunks - 1;
        const int qj = kFp8 ? (rope ? kQChunks - 1 : 0) : j;   // the barrier of this chunk's query
        if (flags & kFirst) ok = wait(ctl.q_full[qj], item & 1);
        if (ok && j > 0) ok = wait(ctl.full[slot], phase);
        if (!ok) break;
        tc_fence_after();
        const uint64_t ad = ring_desc + (uint32_t)slot * (kSlot >> 4);
        const uint64_t bd = q_desc + (uint32_t)(rope ? kQChunks - 1 : j) * (q_chunk >> 4);
        if (leader) {
          if (kFp8 && !rope) {
            const uint64_t lo = bd + 4 * (q_chunk >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {   // hi then lo into the same accumulator
              mma_f8_ss(d, ad + 2 * kk, bd + 2 * kk, idesc8, (j | kk) ? 1u : 0u);
              mma_f8_ss(d, ad + 2 * kk, lo + 2 * kk, idesc8lo, 1u);
            }
          } else {
            const uint32_t dd = kFp8 ? d + kGroupRows : d;   // e4m3: RoPE scores in their own columns
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_ss(dd, ad + 2 * kk, bd + 2 * kk, idesc16, (kFp8 ? kk : j | kk) ? 1u : 0u);
          }
          mma_commit(smem_u32(&ctl.empty[slot]));
          // the query's chunk is free for the next item (e4m3: the latent part is when the sums are done)
          if ((flags & kLast) && (!kFp8 || rope)) mma_commit(smem_u32(&ctl.q_empty[rope ? kQChunks - 1 : j]));
          if (rope) mma_commit(smem_u32(&ctl.acc_full[u & 1]));
        }
        if (++slot == slots) {
          slot = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
      if (flags & kLast) ++item;
      ++u;
    }
    int dummy = 0;
    if (leader) mma_commit(smem_u32(&ctl.drain));
    __syncwarp();
    mbar_wait<false>(smem_u32(&ctl.drain), 0, &dummy, drain_ns);
    if (!ok && lane == 0) set_status(a.status, MLA_ERR_TIMEOUT);
  } else {
    // ---------------------------------------------------------------- sums (thread = token)
    // Two sets of four warps take the tiles of even and odd number, so that one set's TMEM loads and
    // exponentials overlap the other's; a token is always one thread's.
    const int tr = threadIdx.x & 127, set = threadIdx.x >> 7;   // tr: TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const float qnan = __uint_as_float(0x7FC00000u);
    const unsigned long long scale2 = f2_pack(a.scale_log2, a.scale_log2);
    uint32_t u = 0;
    bool ok = true;
    for_items([&](int b, int Lc, int g, int t0, int t1) {
      const int s_first = g * kGroupRows / a.H;   // query token of the group's first row
      // all sum warps are done with the previous item's rows
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (set == 0) {
        const int row = g * kGroupRows + tr;
        const bool valid = row < a.rows && tr < N;
        ctl.nl2[tr] = valid ? -__ldg(m.lse + (size_t)b * a.rows + row) * kLog2e : -INFINITY;
        ctl.late[tr] = valid ? (uint8_t)(row / a.H - s_first) : 0;
      }
      if constexpr (kFp8) {
        // the group's query in two terms. Its last readers were the previous item's MMAs, and their last
        // sums are done.
        constexpr int kU = 4;   // rows in flight per warp (8, or 4 ahead of 4: registers and code, slower)
        for (int r0 = kU * warp; r0 < N; r0 += 8 * kU) {
          uint4 v[kU][2];
#pragma unroll
          for (int i = 0; i < kU; ++i) {
            const int row = g * kGroupRows + r0 + i;
            const uint4* src = reinterpret_cast<const uint4*>((const uint16_t*)a.q_lat +
                                                             ((size_t)b * a.rows + row) * kR) + 2 * lane;
            v[i][0] = row < a.rows ? __ldg(src) : make_uint4(0u, 0u, 0u, 0u);
            v[i][1] = row < a.rows ? __ldg(src + 1) : make_uint4(0u, 0u, 0u, 0u);
          }
#pragma unroll
          for (int i = 0; i < kU; ++i) {
            const uint32_t w[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w, v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
            uint32_t hi[4], lo[4];
            const uint32_t up = split_row(w, hi, lo);
            const int r = r0 + i;
            // lane's 16 channels: 16-byte piece lane % 8 of the row in chunk lane / 8, 128-byte swizzle
            uint8_t* dst = gQ + (lane >> 3) * q_chunk + r * 128 + (((lane & 7) ^ (r & 7)) << 4);
            *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(dst + 4 * q_chunk) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            if (lane == 0) ctl.a2[r] = __uint_as_float(up << 23) * a.scale_log2;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl.q_full[0]));
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const int least = Lc - a.Sq + 1 + s_first;   // causal: every row of the group sees the tokens before this one
      for (int t = t0; t < t1; ++t, ++u) {
        if ((t & 1) != set) continue;
        const int tok = t * kTile + tr;
        const bool mine = tok < Lc;
        float* out = m.mass + (size_t)b * m.max_seq_len + tok;
        float before = 0.f, ks = 0.f;
        bool good = true;
        if (mine) {
          const int blk = __ldg(a.block_table + (size_t)b * a.max_blocks + tok / kBS);
          good = blk >= 0 && blk < a.num_blocks;
          if (!good) set_status(a.status, MLA_ERR_BAD_BLOCK_ID);
          if (kFp8 && good) ks = __ldg(a.kv_scale + (size_t)blk * kBS + tok % kBS);
          // group 0 starts from mass_in, the others from what this thread stored for the group before
          if (g > 0)
            before = *out;
          else if (m.mass_in)
            before = m.mass_in[(size_t)b * m.max_seq_len + tok];
        }
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait<false>(smem_u32(&ctl.acc_full[u & 1]), (u >> 1) & 1, abort, timeout_ns));
        if (!ok) {   // a wait ran out: the tokens left become NaN
          if (mine) *out = qnan;
          continue;
        }
        tc_fence_after();
        const uint32_t d = tmem + lane_off + (u & 1) * kAccCols;
        const bool masked = a.causal && (t + 1) * kTile > least;   // (tokens past the length are not stored)
        const unsigned long long ks2 = f2_pack(ks, ks);
        unsigned long long sum[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
        // 16 columns (rows) at a time, the next 16 on their way out of TMEM meanwhile
        uint32_t v[2][16], r[2][16];
        auto fetch = [&](int c, int k) {
          tmem_ld16(d + c, v[k]);
          if constexpr (kFp8) tmem_ld16(d + kGroupRows + c, r[k]);
        };
        auto add = [&](int c, int k) {
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const ulonglong2 nl = *reinterpret_cast<const ulonglong2*>(&ctl.nl2[c + i]);
            ulonglong2 ar = make_ulonglong2(0ull, 0ull);
            if constexpr (kFp8) ar = *reinterpret_cast<const ulonglong2*>(&ctl.a2[c + i]);
            const uint32_t late = *reinterpret_cast<const uint32_t*>(&ctl.late[c + i]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int e = i + 2 * h;
              const unsigned long long vv = f2_pack(__uint_as_float(v[k][e]), __uint_as_float(v[k][e + 1]));
              unsigned long long x;
              if constexpr (kFp8) {
                const unsigned long long rr = f2_pack(__uint_as_float(r[k][e]), __uint_as_float(r[k][e + 1]));
                x = fma2(mul2(vv, ks2), h ? ar.y : ar.x, fma2(rr, scale2, h ? nl.y : nl.x));
              } else {
                x = fma2(vv, scale2, h ? nl.y : nl.x);
              }
              float x0, x1;
              f2_unpack(x, x0, x1);
              if (masked) {
                if (tok >= least + (int)((late >> (16 * h)) & 255u)) x0 = -INFINITY;
                if (tok >= least + (int)((late >> (16 * h + 8)) & 255u)) x1 = -INFINITY;
              }
              sum[h] = add2(sum[h], f2_pack(ex2_approx(x0), ex2_approx(x1)));
            }
          }
        };
        fetch(0, 0);
        tmem_wait_ld();
#pragma unroll 1
        for (int c = 0; c < N; c += 32) {   // N is a multiple of 16
          if (c + 16 < N) fetch(c + 16, 1);
          add(c, 0);
          tmem_wait_ld();
          if (c + 16 >= N) break;
          if (c + 32 < N) fetch(c + 32, 0);
          add(c + 16, 1);
          tmem_wait_ld();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl.acc_empty[u & 1]));
        float p0, p1, p2, p3;
        f2_unpack(sum[0], p0, p1);
        f2_unpack(sum[1], p2, p3);
        if (mine) *out = good ? before + ((p0 + p1) + (p2 + p3)) : qnan;
      }
      return true;
    });
    if (!ok) set_status(a.status, MLA_ERR_TIMEOUT);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------------------- host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = (EncodeTiledFn)p;
  });
  return fn;
}

// [d2][d1][d0] elements of `size` bytes, contiguous; boxes of 128 bytes x `rows`, 128-byte swizzle
bool map_rows(CUtensorMap* tm, const void* base, uint64_t d0, uint64_t d1, uint64_t d2, int size, uint32_t rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {d0 * size, d0 * d1 * size};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / size), rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(tm, size == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool mass_tc_supported(int r, int d_r, int block_size, int q_dtype, int cache_dtype) {
  return r == kR && d_r == kDR && block_size == kBS && q_dtype == kBF16 && (cache_dtype == kBF16 || cache_dtype == kE4M3);
}

cudaError_t launch_mass_tc(const MassArgs& m0, cudaStream_t s) {
  MassArgs m = m0;
  const DecodeArgs& a = m.d;
  const bool fp8 = a.cache_dtype == kE4M3;
  // MMA N: the rows of a group, in steps of 16
  const int N = std::min(kGroupRows, (a.rows + 15) / 16 * 16);
  const uint32_t q_bytes = kQChunks * (uint32_t)N * 128;
  const int slots = (int)std::min<uint32_t>(kMaxSlots, (kSmemMax - 1024 - kCtlBytes - q_bytes) / kSlot);
  const uint32_t smem = 1024 + kCtlBytes + q_bytes + (uint32_t)slots * kSlot;
  CUtensorMap tq, tqr, tkv, tkr;
  if (!map_rows(&tq, a.q_lat, kR, a.rows, a.B, 2, N) || !map_rows(&tqr, a.q_rope, kDR, a.rows, a.B, 2, N) ||
      !(fp8 ? map_rows(&tkv, a.cache, kR, kBS, a.num_blocks, 1, kBS) && map_rows(&tkr, a.k_rope, kDR, kBS, a.num_blocks, 2, kBS)
            : map_rows(&tkv, a.cache, kR + kDR, kBS, a.num_blocks, 2, kBS)))
    return cudaErrorInvalidValue;
  if (!fp8) tkr = tkv;   // unused
  auto kernel = fp8 ? mass_tc_kernel<true> : mass_tc_kernel<false>;
  static std::once_flag once[2][64];
  static int sms[2][64];
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t err = cudaSuccess;
  std::call_once(once[fp8 ? 1 : 0][dev & 63], [&] {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms[fp8 ? 1 : 0][dev & 63], cudaDevAttrMultiProcessorCount, dev);
  });
  if (err != cudaSuccess) return err;
  // one CTA per SM, fewer when there cannot be as many tiles
  const long long most = (long long)a.B * ((a.len_cap + kTile - 1) / kTile);
  if (m.d.W == 0) m.d.W = (int)std::min<long long>(std::max(sms[fp8 ? 1 : 0][dev & 63], 1), std::max(most, 1ll));
  kernel<<<m.d.W, kTcThreads, smem, s>>>(tq, tqr, tkv, tkr, m, N, slots, wait_timeout_ns(), drain_timeout_ns());
  return cudaGetLastError();
}

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
