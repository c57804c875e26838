// Device helpers shared by the decode, combine and probe kernels: storage decoders,
// the sticky status word and the split plan.
#pragma once

#include <cstdint>

#include "mla_internal.h"
#include "ptx_sm100.cuh"
#include "../../include/mla_decode.h"

namespace mla {

__device__ __forceinline__ void set_status(int* status, int code) {
  if (*((volatile int*)status) == 0) atomicCAS(status, 0, code);
}

__device__ __forceinline__ float bf16_bits_to_float(uint16_t b) {
  return __uint_as_float((uint32_t)b << 16);
}

// OCP FP8 e4m3 (1 sign, 4 exponent bits with bias 7, 3 mantissa bits, no infinities,
// S.1111.111 = NaN) to fp32, written from that definition. Every code is exact in fp32.
__device__ __forceinline__ float e4m3_to_float(uint32_t code) {
  const uint32_t e = (code >> 3) & 0xF, m = code & 0x7;
  float v;
  if (e == 0)
    v = (float)m * 0x1p-9f;                                    // subnormal: m/8 * 2^-6
  else if (e == 0xF && m == 0x7)
    v = __uint_as_float(0x7FC00000u);                          // NaN
  else
    v = __uint_as_float(((e + 120u) << 23) | (m << 20));       // (1 + m/8) * 2^(e-7)
  return (code & 0x80) ? -v : v;
}

// A bf16 row as an e4m3 and an e5m2 row, so that the FP8 tensor path multiplies it: x * 2^-e = hi + lo, with
// one e per row chosen so that its largest magnitude lands in [128, 256). hi is the nearest e4m3 value (4
// significant bits), lo the remainder behind it, in e5m2. A bf16 value has 8 significant bits, so the remainder
// is 0 to 8 of its last places, which e5m2's 3 bits hold: hi + lo is exact from e4m3's smallest normal 2^-6
// upward, 2^-13 of the row's largest magnitude. Below, the remainder is at most 2^-10 and lo off by 2^-14 at
// most: 2^-14 / 128 = 2^-21 of that magnitude.
__device__ __forceinline__ float bf16x2_amax(uint32_t v) {
  return fmaxf(fabsf(__uint_as_float(v << 16)), fabsf(__uint_as_float(v & 0xFFFF0000u)));
}
// e from the row's largest magnitude (taken as at least 2^-100, so that 2^-e stays finite)
__device__ __forceinline__ int split_exponent(float amax) { return max((int)(__float_as_uint(amax) >> 23), 27) - 127 - 7; }

__device__ __forceinline__ uint32_t f32x2_to_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e5m2 codes (2 mantissa bits, normal from 2^-14, smallest step 2^-16).
__device__ __forceinline__ uint32_t f32x2_to_e5m2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// The number c for which (x + c) - c is x to the nearest e4m3 value (|x| below 448): 1.5 * 2^20 times the
// power of two at or below |x|, or times 2^-6, e4m3's smallest normal: c's last place is then that of x's
// four significant bits, and 2^-9 for smaller x. (Arithmetic: conversions there and back run at a quarter
// of its rate or less.)
__device__ __forceinline__ float e4m3_rounder(float x) {
  return __uint_as_float(max(__float_as_uint(x) & 0x7F800000u, 121u << 23) + ((20u << 23) | 0x400000u));
}
// A pair of values (packed, see f2_pack) as two hi codes and two lo codes.
__device__ __forceinline__ void two_terms(unsigned long long x2, uint32_t& hi, uint32_t& lo) {
  const unsigned long long minus = ptx::f2_pack(-1.f, -1.f);
  float x0, x1, h0, h1, l0, l1;
  ptx::f2_unpack(x2, x0, x1);
  const unsigned long long c2 = ptx::f2_pack(e4m3_rounder(x0), e4m3_rounder(x1));
  const unsigned long long h2 = ptx::fma2(c2, minus, ptx::add2(x2, c2));   // hi's value
  ptx::f2_unpack(h2, h0, h1);
  ptx::f2_unpack(ptx::fma2(h2, minus, x2), l0, l1);
  hi = f32x2_to_e4m3(h0, h1);
  lo = f32x2_to_e5m2(l0, l1);
}
// four values (two bf16 pairs) -> four hi codes and four lo codes; down = 2^-e
__device__ __forceinline__ void split_f8(uint32_t v0, uint32_t v1, float down, uint32_t& hi, uint32_t& lo) {
  const unsigned long long d2 = ptx::f2_pack(down, down);
  uint32_t h[2], l[2];
  two_terms(ptx::mul2(ptx::f2_pack(__uint_as_float(v0 << 16), __uint_as_float(v0 & 0xFFFF0000u)), d2), h[0], l[0]);
  two_terms(ptx::mul2(ptx::f2_pack(__uint_as_float(v1 << 16), __uint_as_float(v1 & 0xFFFF0000u)), d2), h[1], l[1]);
  hi = h[0] | (h[1] << 16);
  lo = l[0] | (l[1] << 16);
}

__device__ __forceinline__ float load_q(const void* p, int dtype, size_t i) {
  return dtype == kF32 ? __ldg((const float*)p + i) : bf16_bits_to_float(__ldg((const uint16_t*)p + i));
}

// ---------------------------------------------------------------------------- plan
//
// The work of one call is the batch-ordered list of every sequence's cache blocks
// ("tiles"): T = sum_b ceil(L_b / bs). With W' = min(W, T) active workers, worker
// w < W' owns tiles [floor(w T / W'), floor((w + 1) T / W')): at least one tile each,
// so the workers that touch a sequence are consecutive. The part of sequence b that
// worker w owns is one split; the splits of b are numbered from the first worker that
// touches b, and the split's partial result goes to workspace slot w + b.

__device__ __forceinline__ int clamp_len(int L, int cap, int* status) {
  if (L < 0 || L > cap) {
    set_status(status, MLA_ERR_BAD_SEQ_LEN);
    return L < 0 ? 0 : cap;
  }
  return L;
}

__device__ __forceinline__ int tiles_of(int Lc, int bs) { return (Lc + bs - 1) / bs; }

// Worker containing flat tile x (largest w with floor(w T / W) <= x).
__device__ __forceinline__ int worker_of_tile(long long x, long long T, int W) {
  return (int)(((x + 1) * (long long)W - 1) / T);
}

// Which cache blocks of a sequence make up its tile list.
//   DenseTiles: all of them, tile i is block i.
//   WindowTiles: those that hold a token some query row sees through the window or as a sink: the
//     blocks of tokens [0, min(sinks, L)), then those of [lo, L), lo = the first token of the
//     first row's window. Tile i is block i before the gap and i + gap behind it.
struct DenseTiles {
  static constexpr bool kCuts = false;   // never aligned to sequences (see cut() below)
  int bs;
  __device__ __forceinline__ DenseTiles(int bs_) : bs(bs_) {}
  __device__ __forceinline__ int count(int Lc) const { return tiles_of(Lc, bs); }
  __device__ __forceinline__ int block(int i, int) const { return i; }
  __device__ __forceinline__ int gap(int) const { return 0; }
};

struct WindowTiles {
  static constexpr bool kCuts = true;
  int bs, Sq, causal, window, sinks, aligned;
  __device__ __forceinline__ WindowTiles(const DecodeArgs& a)
      : bs(a.bs), Sq(a.Sq), causal(a.causal), window(a.window), sinks(a.sinks), aligned(a.aligned) {}
  // first token of the earliest window among the sequence's query rows
  __device__ __forceinline__ int lo(int Lc) const {
    const int first = causal ? max(Lc - Sq + 1, 0) : Lc;
    return max(first - window, 0);
  }
  __device__ __forceinline__ int sink_tiles(int Lc) const { return tiles_of(min(sinks, Lc), bs); }
  __device__ __forceinline__ int gap(int Lc) const { return max(lo(Lc) / bs - sink_tiles(Lc), 0); }
  __device__ __forceinline__ int count(int Lc) const { return tiles_of(Lc, bs) - gap(Lc); }
  __device__ __forceinline__ int block(int i, int Lc) const { return i < sink_tiles(Lc) ? i : i + gap(Lc); }
  // How the tile list is cut among the workers: k > 0 sequences per worker, -k > 0 workers per sequence, or
  // 0: evenly, wherever that falls (see WorkerPlan). A window's tile lists are short and nearly all alike, and
  // a worker's second segment costs as much as 10 to 20 tiles (its query, the drained pipeline, the
  // epilogue), so cuts at the sequences' ends are worth a longer share; whole sequences have no partial
  // outputs and nothing to merge besides. Measured on 74 workers, 128 rows, bf16, us (even cut, whole,
  // parts), n sequences x tiles:
  //   a few sequences, parts of at least 4 tiles: 1 x 33: 39, 55, 33; 9 x 33: 44, 56, 36; 3 x 9: 31, 31, 31
  //   (e4m3 39, 46, 39);
  //   two to four workers per sequence: 32 x 9: 47, 33, 39 (e4m3 65, 47, 49); 16 x 17: 45, 39, 36;
  //   32 x 17: 54, 41, 43 (e4m3 74, 61, 56); 32 x 65: 84, 93, 74;
  //   a longest share 12 tiles above the even one: 15 x 257: 109, -, 109;
  //   one worker or less per sequence: 64 x 65: 129, 111; 40 x 33: 77, 70; 80 x 8: 67, 57; 80 x 17: 80, 81.
  // The same thresholds serve fewer rows and the e4m3 cache. Over 28 such batches (1 to 300 sequences, windows of 60
  // to 4096) with 8 and 128 rows, bf16 and e4m3, the even cut takes 0.84 to 1.38 times this rule's time, 1.08 in the
  // mean: 70 x 8 e4m3 1.30 (8 rows), 1.28 (128); 300 x 2 1.00, 1.38; but 80 x 17 0.84 (8 rows, 0.98 with 128), where
  // few rows leave no merge to save, and 50 x 65 0.89, 0.98.
  // Where nothing is hidden the cut stays the dense one, and with it the result.
  __device__ __forceinline__ int cut(long long T, int most, int hidden, int B, int W) const {
    if (!aligned || hidden == 0) return 0;
    const int k = (B + W - 1) / W, p = min(min(W / B, (most + 3) / 4), 32);
    if (p > 1) {
      const int share = (most + p - 1) / p;
      if (most - share > 5) return share <= T / W + 12 ? -p : 0;
    }
    const int more = T <= 2 * W ? 12 : k == 1 ? 22 : 16;
    return (long long)k * most <= T / W + more ? k : 0;
  }
};

template <bool kWindow>
struct TilesOf {
  typedef DenseTiles type;
  static __device__ __forceinline__ DenseTiles make(const DecodeArgs& a) { return DenseTiles(a.bs); }
};
template <>
struct TilesOf<true> {
  typedef WindowTiles type;
  static __device__ __forceinline__ WindowTiles make(const DecodeArgs& a) { return WindowTiles(a); }
};

// The columns of a tile's slice [base, base + n) of tokens that a query row with n_row tokens sees:
// [0, sink) and [first, end).
struct WindowCols {
  int sink, first, end;
  __device__ __forceinline__ WindowCols(const DecodeArgs& a, int n_row, int base, int n)
      : sink(min(max(min(a.sinks, n_row) - base, 0), n)),
        first(min(max(n_row - a.window - base, 0), n)),
        end(min(max(n_row - base, 0), n)) {}
  __device__ __forceinline__ bool all(int n) const { return end == n && (first == 0 || sink == n); }
  __device__ __forceinline__ bool sees(int j) const { return j < end && (j >= first || j < sink); }
};

//
// When tiles.cut() says so, workers are aligned to sequences instead: worker w owns sequences
// [k w, k (w + 1)) whole (k > 0), or part w % p of sequence w / p (p = -k > 0 workers each, of which the
// first min(p, tiles) have a part).

struct WorkerPlan {
  long long T;      // total tiles
  int W;            // active workers, min(W, T)
  int cut;          // sequences per worker, -(workers per sequence), or 0: the even cut
  long long start;  // first tile of this worker (workers per sequence: its part)
  long long end;    // one past its last tile (aligned to sequences: one past its last sequence)
  long long P0;     // flat index of sequence b0's first tile
  int b0;           // first sequence with a tile in [start, end)
};

// Executed by one full warp; every lane returns the same plan.
template <class Tiles>
__device__ __forceinline__ WorkerPlan warp_plan(const int32_t* __restrict__ seq_lens, int B, const Tiles& tiles,
                                                int cap, int W, int w, int* status) {
  const int lane = threadIdx.x & 31;
  long long T = 0;
  int most = 0, hidden = 0;
  for (int b = lane; b < B; b += 32) {
    const int Lc = clamp_len(__ldg(seq_lens + b), cap, status), n = tiles.count(Lc);
    T += n;
    most = max(most, n);
    hidden = max(hidden, tiles.gap(Lc));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) T += __shfl_xor_sync(0xffffffffu, T, o);
  WorkerPlan p;
  p.T = T;
  p.W = (T > 0 && T < W) ? (int)T : W;
  p.cut = 0;
  if constexpr (Tiles::kCuts) {
    most = __reduce_max_sync(0xffffffffu, most);
    hidden = __reduce_max_sync(0xffffffffu, hidden);
    p.cut = tiles.cut(T, most, hidden, B, W);
    if (p.cut) {
      const int parts = max(-p.cut, 1), k = max(p.cut, 1);   // one of them is 1
      p.W = W;
      p.b0 = (int)min((long long)(w / parts) * k, (long long)B);
      p.start = w % parts;
      p.P0 = 0;
      p.end = min((long long)(w / parts + 1) * k, (long long)B);
      return p;
    }
  }
  p.start = (T > 0 && w < p.W) ? (long long)w * T / p.W : T;
  p.end = (T > 0 && w < p.W) ? (long long)(w + 1) * T / p.W : T;
  p.b0 = B;
  p.P0 = T;
  if (p.start >= p.end) return p;
  long long carry = 0;
  for (int base = 0; base < B; base += 32) {
    const int b = base + lane;
    const int n = b < B ? tiles.count(clamp_len(__ldg(seq_lens + b), cap, status)) : 0;
    long long incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const long long P = carry + incl - n;
    const bool hit = n > 0 && P <= p.start && p.start < P + n;
    const unsigned m = __ballot_sync(0xffffffffu, hit);
    if (m) {
      const int src = __ffs(m) - 1;
      p.b0 = base + src;
      p.P0 = __shfl_sync(0xffffffffu, P, src);
      return p;
    }
    carry += __shfl_sync(0xffffffffu, incl, 31);
  }
  return p;
}

__device__ __forceinline__ WorkerPlan warp_plan(const int32_t* __restrict__ seq_lens, int B, int bs,
                                                int cap, int W, int w, int* status) {
  return warp_plan(seq_lens, B, DenseTiles(bs), cap, W, w, status);
}

// One split of a sequence as seen by its worker.
struct Segment {
  int b;
  int tile_begin, tile_end;   // range of sequence b's tile list
  int first_worker, splits;   // workers touching b
  int split;                  // this worker's index among them
  int Lc;                     // clamped sequence length
};

// Iterates the segments of a worker's range. Usage:
//   SegmentIter it(plan, ...); Segment sg; while (it.next(sg)) { ... }
template <class Tiles>
struct SegmentIterT {
  const int32_t* seq_lens;
  Tiles tiles;
  int B, cap, W, w;
  int* status;
  WorkerPlan p;
  int b;
  long long P;

  __device__ SegmentIterT(const WorkerPlan& plan, const int32_t* sl, int B_, const Tiles& t, int cap_, int w_, int* st)
      : seq_lens(sl), tiles(t), B(B_), cap(cap_), W(plan.W), w(w_), status(st), p(plan), b(plan.b0), P(plan.P0) {}

  __device__ bool next(Segment& sg) {
    if constexpr (Tiles::kCuts) {
      while (p.cut && b < (int)p.end) {
        sg.Lc = clamp_len(__ldg(seq_lens + b), cap, status);
        sg.b = b++;
        const int n = tiles.count(sg.Lc);
        sg.split = (int)p.start;
        sg.first_worker = w - sg.split;
        sg.splits = min(max(-p.cut, 1), n);
        if (sg.split >= sg.splits) continue;   // (no tile at all among them)
        sg.tile_begin = (int)((long long)n * sg.split / sg.splits);
        sg.tile_end = (int)((long long)n * (sg.split + 1) / sg.splits);
        return true;
      }
      if (p.cut) return false;
    }
    while (b < B && P < p.end) {
      const int Lc = clamp_len(__ldg(seq_lens + b), cap, status);
      const int n = tiles.count(Lc);
      const int cur = b++;
      const long long Pb = P;
      P += n;
      if (n == 0) continue;
      const long long s0 = Pb > p.start ? Pb : p.start;
      const long long s1 = (Pb + n) < p.end ? (Pb + n) : p.end;
      if (s1 <= s0) continue;
      sg.b = cur;
      sg.tile_begin = (int)(s0 - Pb);
      sg.tile_end = (int)(s1 - Pb);
      sg.first_worker = worker_of_tile(Pb, p.T, W);
      sg.splits = worker_of_tile(Pb + n - 1, p.T, W) - sg.first_worker + 1;
      sg.split = w - sg.first_worker;
      sg.Lc = Lc;
      return true;
    }
    return false;
  }
};

using SegmentIter = SegmentIterT<DenseTiles>;

// Physical block of tile `tile` of sequence b, validated (bad ids read block 0).
__device__ __forceinline__ int checked_block(const int32_t* __restrict__ bt, int max_blocks, int b, int tile,
                                             int num_blocks, int* status) {
  int blk = __ldg(bt + (size_t)b * max_blocks + tile);
  if (blk < 0 || blk >= num_blocks) {
    set_status(status, MLA_ERR_BAD_BLOCK_ID);
    blk = 0;
  }
  return blk;
}

// Warp-collective: the part of sequence b in tiles [t0, t1) read something it may not: the
// sequence's length is out of range, a block id is out of range, or (sparse decode, sel_idx set)
// a listed position is outside the block table or maps to a bad block. Such rows are written as
// NaN.
template <class Tiles>
__device__ __forceinline__ bool segment_poisoned(const DecodeArgs& a, const Tiles& tiles, int b, int t0, int t1) {
  const int lane = threadIdx.x & 31;
  const int L = __ldg(a.seq_lens + b);
  bool bad = L < 0 || L > a.len_cap;
  if (a.sel_idx == nullptr) {
    for (int t = t0 + lane; t < t1; t += 32) {
      const int Lc = min(max(L, 0), a.len_cap);
      const int blk = __ldg(a.block_table + (size_t)b * a.max_blocks + tiles.block(t, Lc));
      bad |= blk < 0 || blk >= a.num_blocks;
    }
  } else if (!bad) {
    const int pos_cap = a.max_blocks * a.bs;
    const int j1 = min(t1 * a.bs, L);
    for (int j = t0 * a.bs + lane; j < j1; j += 32) {
      const int t = __ldg(a.sel_idx + (size_t)b * a.top_k + j);
      const int blk = (t >= 0 && t < pos_cap) ? __ldg(a.block_table + (size_t)b * a.max_blocks + t / a.bs) : -1;
      bad |= blk < 0 || blk >= a.num_blocks;
    }
  }
  return __any_sync(0xffffffffu, bad);
}

}  // namespace mla
