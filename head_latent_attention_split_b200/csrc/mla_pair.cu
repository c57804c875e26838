// Split-role tensor-core (tcgen05 + TMA) absorbed-MLA decode for r = 512, d_r = 64, 64-token
// cache blocks, bf16 queries and a bf16 cache; dense token ranges, or (kSparse) each sequence's
// list of selected positions.
//
// The fp32 output of 128 query rows over all 512 latent channels, O[128 x 512], fills the 512
// TMEM columns of one SM, so a decode worker is a cluster of two CTAs. The roles differ:
//
//   score CTA (cluster rank 0): streams every tile of the worker's range whole (512 latent +
//     64 RoPE channels) and computes full scores S = Q . C^T with tcgen05: A = the absorbed
//     query held in TMEM, B = the cache rows in shared memory. Tiles are scored two at a time
//     (N = 128 tokens per MMA): on B200 a tcgen05 MMA costs ~60 cycles up to N = 64 and ~70 at
//     N = 128, so pairs of tiles nearly double the score rate. The cache ring is 3 slots of
//     48 KB, each three 64-channel chunks of both tiles of a pair (6 TMA boxes per barrier).
//     Eight softmax warps (two per SM sub-partition: warp q takes the first tile's 64 columns
//     of rows [32q, 32q + 32), warp q + 4 the second tile's) run the online softmax in
//     registers, thread = query row, share the row maximum through shared memory, and write
//     each tile's message (bf16 P[128 x 64] as K-major core matrices plus one rescale factor
//     and 1/row-sum per row, 17 KB) into one of four staging buffers; a post warp sends each
//     message with one bulk copy into the output CTA's shared memory.
//   output CTA (cluster rank 1): streams the same tiles' 512 latent channels (one 4-D TMA box per
//     256 channels; the second read of each tile is served by L2), rescales O rows whose
//     running maximum moved, and accumulates O[128 x 512] += P . C with tcgen05 (A = P in
//     shared memory, B = the tile read N-major, N = 256), then normalises O into the output
//     (or the split partial).
//
// Only P crosses between the SMs, in one direction. The completion of the PV that read a
// receive buffer is signalled straight to the score CTA by the tensor core (a commit arriving on
// the score CTA's barrier), and the output CTA hands a staging buffer back with one remote
// arrive once its message has landed, so no thread waits on a round trip per tile.
//
// The running maximum of a row only moves when a tile pair raises it by more than 2^8 (log2
// units), so O is rescaled rarely; the softmax uses base-2 exponentials of scale * log2(e) *
// score. Work split over workers: the flat block-list plan of mla_device.cuh (same as every
// kernel); pairs never straddle two sequences (a sequence with an odd number of tiles ends with
// a single tile, scored with N = 64). Every wait is bounded; a timeout sets MLA_ERR_TIMEOUT and
// the rows of the unfinished segments are written as NaN.
//
// kFp8 (window decode over an e4m3 cache): the codes are MMA operands as they are, in both CTAs; nothing
// is converted per tile.
//   scores: the query is split into an e4m3 and an e5m2 term (split_f8) that fill 256 TMEM columns; both multiply
//     every 128-channel chunk of codes into one accumulator, and the RoPE parts (bf16, the query's in
//     shared memory) have a second one, since a token's scale applies to the latent part only:
//     score = 2^e (acc s_t + rope), the query's power of two in the row's softmax scale. e is the latent part's
//     (its terms are what has few bits), unless the RoPE part, in bf16, is 2^64 times as large. 36 MMAs per tile
//     pair, as with a bf16 cache.
//   probabilities: w = P s_t as hi = e4m3(w) and lo = e5m2(w - hi), the remainder behind the stored hi, so the
//     PV is 8 MMAs per tile on the codes themselves. The remainder of 4 significant bits is at most half of
//     the fourth one, and e5m2's three hold it to 2^-8 of w, a bf16 rounding's accuracy, from e4m3's smallest
//     normal 2^-6 upward; a smaller w is off by 2^-14 at most (remainders up to half of e4m3's step 2^-9).
//     What that loses must stay small against the row's sum however many tokens there are (a sink that holds
//     half of it leaves every other token 2^-14 and less), so the reference of w follows the maximum of score
//     + log2 s_t, the logarithm of what w holds, up AND down: it is set 2^4 below a pair's maximum when that
//     exceeds it by 2^8, and again, by the largest of them, when eight pairs of one row stayed below
//     2^2. Per reference the pairs below 2^2 lose 8 x 128 x 2^-14 = 2^-4 at most, against the token of 2^4
//     that set it, and any other pair 128 x 2^-14 = 2^-7 against its own maximum of 2^2 or more: together
//     2^-8 + 2^-9 of the row's sum of w, for any scores and any length. (The reference goes down by 2^24
//     below its highest at most, so that sums stay finite; what is smaller than that has no weight.)
//     Down steps cost what the up steps do, a pass over O: at scores of deviation 1.7, 33 pairs make 6 up and
//     2 down steps per warp.
//   Half the bytes per tile: twice the ring slots.
//   Bound by the softmax warps, 3.3 us per tile pair at 128 rows (bf16 2.3): scores and scales 1.1,
//   exponentials and the two terms 1.3, the message 0.55, the rest waiting; a segment's start costs
//   another 11 us, most of it the query's split.
//
// kWindow: the tile list holds only the blocks that some row sees (WindowTiles), the softmax masks what a
// row does not see of them, and the cut among the workers is WindowTiles::cut's. 128 heads, bf16: 64
// sequences x 65 tiles in 100 us (3.1 TB/s of cache, 42 % of the tensor pipe's time); 96 sequences x 256 causal
// rows, windows of 1500: 132 us; e4m3, 32 x 33 tiles: 74 us. Bound by the coupled latencies of the tile loop
// (2.3 us per pair, of which the 36 score MMAs 1.4) and by a segment's 14 us around it.
#include <cuda.h>

#include <cmath>
#include <mutex>

#include "mla_device.cuh"
#include "mla_tc.h"
#include "ptx_sm100.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kR = 512, kDR = 64, kBS = 64, kRows = 128;
constexpr uint32_t kChunk = kBS * 128;                 // [64 tok][64 ch] bf16, 128-byte swizzle
constexpr uint32_t kDChunk = 2 * kChunk;               // one chunk of both tiles of a pair
constexpr int kChunksS = 9;                            // score CTA: 8 latent chunks + the RoPE chunk
constexpr int kGroupS = 3;                             // score CTA: double chunks per ring slot (6 boxes)
constexpr uint32_t kSlotBytesS = kGroupS * kDChunk;    // 48 KB
constexpr int kSlotsS = 3;                             // score CTA ring of slots
constexpr uint32_t kHalf = 4 * kChunk;                 // output CTA half stage: 256 channels of a tile
constexpr int kHalvesO = 5;                            // output CTA ring of half stages
// e4m3 cache: slots of one chunk (128 channels of codes, or the RoPE keys, of both tiles), half stages of
// two chunks
constexpr int kChunksS8 = 5, kSlotsS8 = 8, kHalvesO8 = 10;
constexpr uint32_t kSlotBytesS8 = kDChunk, kHalf8 = 2 * kChunk;
constexpr uint32_t kPBytes = kRows * 128;              // P [128 rows][64 tokens] bf16
constexpr uint32_t kMsgBytes = kPBytes + kRows * 8;    // + (rescale factor, 1 / row sum) per row
constexpr int kStage = 4;                              // score CTA: outgoing message buffers
constexpr int kRxBufs = 3;                             // output CTA: receive buffers

constexpr uint32_t kOffRingS = 0;
constexpr uint32_t kOffStage = kOffRingS + kSlotsS * kSlotBytesS;   // score CTA: outgoing messages
constexpr uint32_t kOffRx = 0;                         // output CTA: messages of the tiles in flight
constexpr uint32_t kOffRingO = kOffRx + kRxBufs * kMsgBytes;
constexpr uint32_t kEndS = kOffStage + kStage * kMsgBytes, kEndO = kOffRingO + kHalvesO * kHalf;
constexpr uint32_t kOffCtl = (kEndS > kEndO ? kEndS : kEndO);
constexpr uint32_t kSmemBytes = kOffCtl + 4096 + 1024;     // control block + alignment slack
// e4m3 cache: the query's RoPE part [128 rows][64] bf16, then the messages; behind the control block the
// token scales of four pairs, each softmax warp's 64 logarithms of them and 64 finite copies, the halves'
// query maxima
constexpr uint32_t kOffQr8 = kSlotsS8 * kSlotBytesS8, kOffStage8 = kOffQr8 + kRows * 128;
constexpr uint32_t kOffScale8 = kOffCtl + 4096, kOffLog8 = kOffScale8 + 4 * 128 * 4, kOffQmax8 = kOffLog8 + 8 * 128 * 4;
constexpr uint32_t kSmemBytes8 = kOffQmax8 + 2 * kRows * 4 + 1024;
static_assert(kOffStage8 + kStage * kMsgBytes <= kOffCtl && kOffRx + kRxBufs * kMsgBytes + kHalvesO8 * kHalf8 <= kOffCtl &&
                  kSmemBytes8 <= 232448,
              "e4m3 layout");
static_assert(kSlotBytesS % 1024 == 0 && kOffRingO % 1024 == 0 && kMsgBytes % 1024 == 0 && kOffCtl % 1024 == 0,
              "swizzled buffers need 1024-byte alignment");
static_assert(kSmemBytes <= 232448, "shared memory budget");

// TMEM columns. Score CTA: the absorbed query (bf16 pairs, 288 columns = 576 channels) and one
// score buffer of 128 columns (a tile pair); output CTA: O.
constexpr uint32_t kTmemQ = 0;
constexpr uint32_t kTmemS = 288;
constexpr uint32_t kTmemCols = 512;
static_assert(kTmemS + 128 <= kTmemCols, "TMEM budget of the score CTA");
// e4m3 cache: the query's hi terms (128 columns) and lo terms (128), the latent and the RoPE scores
constexpr uint32_t kTmemLo8 = 128, kTmemS8 = 256, kTmemR8 = 384;

constexpr int kRowThreads = 256;   // warps 0-7: softmax (score CTA) / row work (output CTA)
constexpr int kThreads = kRowThreads + 96;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kPostWarp = 10;      // score CTA: copies each written message to the output CTA
constexpr float kRescaleThreshold = 8.0f;
// e4m3 cache: P s_t starts at 2^4 and stays below 2^8; pairs whose maximum is below 2^2 lower the reference when
// there are kLowPairs8 of them, to 2^-24 of its highest at most
constexpr float kHeadroom8 = 4.0f, kLow8 = 2.0f, kDepth8 = 24.0f;
constexpr int kLowPairs8 = 8;
constexpr float kScaleFloor = 0x1p-64f;   // of a token's scale, in the running maximum only

struct Ctl {
  // score CTA
  uint64_t full[kSlotsS8], empty[kSlotsS8];
  uint64_t q_full, q_empty;
  uint64_t s_full, s_empty;
  uint64_t written[kStage];     // the 128 softmax threads of a tile wrote its message into buffer s
  uint64_t sent[kStage];        // the message in buffer s reached the output CTA (s is free again)
  uint64_t credit[kRxBufs];     // the output CTA's PV that read receive buffer b has completed
  // output CTA
  uint64_t ofull[kHalvesO8], oempty[kHalvesO8];
  uint64_t rx_full[kRxBufs];    // the message of a tile landed in receive buffer b
  uint64_t p_ready[kRxBufs];    // rows of buffer b checked (rescaled, tail zeroed): PV may run
  uint64_t pv_done[kRxBufs];
  uint64_t drain;
  uint64_t xbar[4];          // score CTA: the two softmax warps of lane quarter q posted their maxima
  uint64_t sbar[4];          // ... their row sums (a segment's last pair)
  uint64_t qbar[4];          // ... e4m3 cache: their rows' query maxima
  uint64_t sc_full[4];       // e4m3 cache: the token scales of pair u landed in slot u % 4
  uint32_t tmem_base;
  int abort;
  WorkerPlan plan;
  float xmax[2][2][kRows];   // score CTA: [pair parity][column half][row] partial row maxima
  float xsum[2][kRows];      // score CTA: [column half][row] row sums at a segment's end
};
static_assert(sizeof(Ctl) <= 4096, "control block");

// One arrival for the whole warp, after every lane's earlier memory operations (the barriers
// that warps 0-7 signal count warps, not threads).
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Physical block of tile `tile` of sequence b; an id out of range sets the status word and
// maps to the block just past the cache, which TMA reads as zeros.
__device__ __forceinline__ int tile_block(const DecodeArgs& a, int b, int tile) {
  const int blk = __ldg(a.block_table + (size_t)b * a.max_blocks + tile);
  if (blk < 0 || blk >= a.num_blocks) {
    set_status(a.status, MLA_ERR_BAD_BLOCK_ID);
    return a.num_blocks;
  }
  return blk;
}

// Prefetch into L2 the query rows of row group rg of sequence b (latent and RoPE parts), so the
// softmax warps' loads of a new segment's query hit L2: the score MMAs wait for them.
__device__ __forceinline__ void prefetch_query(const DecodeArgs& a, int b, int rg) {
  const int r0 = rg * kRows, nr = min(kRows, a.rows - r0);
  if (nr <= 0) return;
  const size_t row = (size_t)b * a.rows + r0;
  prefetch_l2((const uint16_t*)a.q_lat + row * kR, (uint32_t)nr * kR * 2);
  prefetch_l2((const uint16_t*)a.q_rope + row * kDR, (uint32_t)nr * kDR * 2);
}

// Physical cache row of entry j of sequence b's selected-token list (sparse decode). Entries
// past the count, and entries whose position or block id is out of range (which also sets the
// status word), map to the row just past the cache, which the row gathers read as zeros.
__device__ __forceinline__ int sparse_row(const DecodeArgs& a, int b, int j, int count) {
  const int oob = a.num_blocks * kBS;
  if (j >= count) return oob;
  const int t = __ldg(a.sel_idx + (size_t)b * a.top_k + j);
  const int blk = (t >= 0 && t < a.max_blocks * kBS) ? __ldg(a.block_table + (size_t)b * a.max_blocks + t / kBS) : -1;
  if (blk < 0 || blk >= a.num_blocks) {
    set_status(a.status, MLA_ERR_BAD_BLOCK_ID);
    return oob;
  }
  return blk * kBS + t % kBS;
}

// kSparse: tile t of a sequence is entries [64 t, 64 t + 64) of its selected-token list (the
// sparse decode); tm_kv is then the cache as rows [num_blocks * 64][576] (one-row boxes of 64
// channels, 128-byte swizzle) and the producers fetch each tile's rows with 4-row gathers.
// kWindow: the tile list holds only the blocks with sink tokens or tokens of the rows' windows
// (WindowTiles); a row's softmax masks the tokens of those blocks that it does not see, and tokens
// that no row sees are zeroed before the PV reads them. The pipelines are the dense ones.
template <bool kSparse, bool kWindow, bool kFp8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    pair_decode_kernel(const __grid_constant__ CUtensorMap tm_kv, const __grid_constant__ CUtensorMap tm_kv4,
                       const __grid_constant__ CUtensorMap tm_kr, const __grid_constant__ CUtensorMap tm_sc,
                       const DecodeArgs a, const int n_rg,
                       const uint64_t timeout_ns, const uint64_t drain_ns) {
  constexpr int kSlots = kFp8 ? kSlotsS8 : kSlotsS, kHalves = kFp8 ? kHalvesO8 : kHalvesO;
  constexpr uint32_t kSlotBytes = kFp8 ? kSlotBytesS8 : kSlotBytesS, kHalfBytes = kFp8 ? kHalf8 : kHalf;
  constexpr uint32_t kOffMsg = kFp8 ? kOffStage8 : kOffStage;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Ctl& ctl = *reinterpret_cast<Ctl*>(smem + kOffCtl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();   // 0: scores and softmax, 1: output
  const uint32_t peer = rank ^ 1u;
  const int cluster = (int)(blockIdx.x >> 1);
  const int w = cluster / n_rg, rg = cluster % n_rg;
  const int cap = a.len_cap;
  volatile int* abort = &ctl.abort;
  typedef SegmentIterT<typename TilesOf<kWindow>::type> SegIter;
  const auto tiles = TilesOf<kWindow>::make(a);
  if constexpr (kWindow) launch_dependents();   // the combine

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_u32(&ctl.full[i]), 1);
      mbar_init(smem_u32(&ctl.empty[i]), 1);
    }
    mbar_init(smem_u32(&ctl.q_full), kRowThreads / 32);   // one arrival per warp
    mbar_init(smem_u32(&ctl.q_empty), 1);
    mbar_init(smem_u32(&ctl.s_full), 1);
    mbar_init(smem_u32(&ctl.s_empty), kRowThreads / 32);
    for (int i = 0; i < kHalves; ++i) {
      mbar_init(smem_u32(&ctl.ofull[i]), 1);
      mbar_init(smem_u32(&ctl.oempty[i]), 1);
    }
    for (int i = 0; i < kStage; ++i) {
      mbar_init(smem_u32(&ctl.written[i]), 4);   // the four warps of one tile
      mbar_init(smem_u32(&ctl.sent[i]), 1);
    }
    for (int i = 0; i < kRxBufs; ++i) {
      mbar_init(smem_u32(&ctl.credit[i]), 1);
      mbar_init(smem_u32(&ctl.rx_full[i]), 1);
      // receive buffers armed for tiles 0 .. kRxBufs - 1
      if (rank == 1) mbar_arrive_expect_tx(smem_u32(&ctl.rx_full[i]), kMsgBytes);
      mbar_init(smem_u32(&ctl.p_ready[i]), kRowThreads / 32);
      mbar_init(smem_u32(&ctl.pv_done[i]), 1);
    }
    mbar_init(smem_u32(&ctl.drain), 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&ctl.xbar[i]), 2);
      mbar_init(smem_u32(&ctl.sbar[i]), 2);
      mbar_init(smem_u32(&ctl.qbar[i]), 2);
      mbar_init(smem_u32(&ctl.sc_full[i]), 1);
    }
    ctl.abort = 0;
    fence_mbarrier_init_cluster();
  }
  if (warp == kProducerWarp) {
    const WorkerPlan p = warp_plan(a.seq_lens, a.B, tiles, cap, a.W, w, a.status);
    if (lane == 0) {
      ctl.plan = p;
      prefetch_tmap(rank == 0 ? &tm_kv : &tm_kv4);
    }
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&ctl.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  cluster_sync();   // both CTAs' barriers initialised, TMEM allocated, plan ready
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  const WorkerPlan plan = ctl.plan;

  auto wait_warp = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait<false>(bar, parity, abort, timeout_ns));
  };

  // Geometry of warps 0-7 (both CTAs): thread = TMEM lane = query row of the group; warp q and
  // q + 4 share the rows of lane quarter q and split the columns (half = warp / 4).
  const int quarter = warp & 3, half = (warp >> 2) & 1;
  const int row = 32 * quarter + lane;
  const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
  const int grow = rg * kRows + row;
  const bool valid_row = grow < a.rows;
  const int s_idx = valid_row ? grow / a.H : 0;

  if (kSparse && rank == 0 && warp == kProducerWarp) {
    // ------------------------------------------------------------------ score CTA: row gathers
    // lane L fetches rows 4L .. 4L + 3 of the tile pair (entries 64 tile + 4L + m), each of the
    // slot's three 64-channel chunks with one 4-row gather: the same slot layout as the tiled
    // loads (second tile's rows right after the first's).
    SegIter it(plan, a.seq_lens, a.B, tiles, cap, w, a.status);
    Segment sg;
    uint32_t c = 0;   // slots issued
    bool ok = true;
    while (ok && it.next(sg)) {
      if (lane == 0) prefetch_query(a, sg.b, rg);
      for (int tile = sg.tile_begin; ok && tile < sg.tile_end; tile += 2) {
        const int nt = min(2, sg.tile_end - tile);
        const bool act = lane < 16 * nt;
        int r4[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) r4[m] = act ? sparse_row(a, sg.b, tile * kBS + 4 * lane + m, sg.Lc) : 0;
#pragma unroll 1   // rolled: see the score MMA loop
        for (int g = 0; g < kChunksS / kGroupS; ++g, ++c) {
          const uint32_t slot = c % kSlots;
          bool free_slot = true;
          if (lane == 0 && c >= (uint32_t)kSlots)
            free_slot = mbar_wait<false>(smem_u32(&ctl.empty[slot]), ((c / kSlots) & 1) ^ 1, abort, timeout_ns);
          ok = __shfl_sync(0xffffffffu, free_slot, 0);
          if (!ok) break;
          const uint32_t bar = smem_u32(&ctl.full[slot]);
          const uint32_t dst = smem_u32(smem + kOffRingS + slot * kSlotBytes);
          if (lane == 0) mbar_arrive_expect_tx(bar, nt * kGroupS * kChunk);
          __syncwarp();
          if (act) {
#pragma unroll
            for (int jj = 0; jj < kGroupS; ++jj)
              tma_gather4(dst + jj * kDChunk + lane * 512, &tm_kv, bar, 64 * (kGroupS * g + jj), r4);
          }
        }
      }
    }
    if (lane == 0) {
      int dummy = 0;
      for (uint32_t i = 0; i < kSlots && i < c; ++i) {
        const uint32_t cl = c - 1 - i;
        mbar_wait<false>(smem_u32(&ctl.full[cl % kSlots]), (cl / kSlots) & 1, &dummy, drain_ns);
      }
      if (!ok) set_status(a.status, MLA_ERR_TIMEOUT);
    }
  } else if (rank == 0 && warp == kProducerWarp) {
    // ------------------------------------------------------------------ score CTA: TMA producer
    if (lane == 0) {
      // (An L2 prefetch of whole blocks a few tiles ahead of these loads measured slower on
      // B200, the farther ahead the slower: the ring's own loads are the only reads.)
      SegIter it(plan, a.seq_lens, a.B, tiles, cap, w, a.status);
      Segment sg;
      uint32_t c = 0, u = 0, sc_issued = 0;   // slots issued, pairs, pairs whose scales are issued
      bool ok = true;
      while (ok && it.next(sg)) {
        prefetch_query(a, sg.b, rg);
        for (int tile = sg.tile_begin; ok && tile < sg.tile_end; tile += 2, ++u) {
          const int nt = min(2, sg.tile_end - tile);
          const int blk0 = tile_block(a, sg.b, tiles.block(tile, sg.Lc));
          const int blk1 = nt == 2 ? tile_block(a, sg.b, tiles.block(tile + 1, sg.Lc)) : 0;
#pragma unroll 1   // rolled: see the score MMA loop
          for (int g = 0; g < (kFp8 ? kChunksS8 : kChunksS / kGroupS); ++g, ++c) {
            const uint32_t slot = c % kSlots;
            if (c >= (uint32_t)kSlots &&
                !mbar_wait<false>(smem_u32(&ctl.empty[slot]), ((c / kSlots) & 1) ^ 1, abort, timeout_ns)) {
              ok = false;
              break;
            }
            const uint32_t bar = smem_u32(&ctl.full[slot]);
            const uint32_t dst = smem_u32(smem + kOffRingS + slot * kSlotBytes);
            if constexpr (kFp8) {
              const bool rope = g == kChunksS8 - 1;
              mbar_arrive_expect_tx(bar, nt * kChunk);
              for (int h = 0; h < nt; ++h)
                tma_load_3d(dst + h * kChunk, rope ? &tm_kr : &tm_kv, bar, rope ? 0 : 128 * g, 0, h ? blk1 : blk0);
              if (rope) {
                // the pair's token scales, into one of four slots: this pair's MMAs cannot run before the
                // softmax warps are done with pair u - 2, nor this load be issued before those of pair u - 2
                const uint32_t sbar = smem_u32(&ctl.sc_full[u & 3]);
                mbar_arrive_expect_tx(sbar, nt * kBS * 4);
                for (int h = 0; h < nt; ++h)
                  tma_load_3d(smem_u32(smem + kOffScale8 + (u & 3) * 512 + h * 256), &tm_sc, sbar, 0, 0, h ? blk1 : blk0);
                ++sc_issued;
              }
            } else {
              mbar_arrive_expect_tx(bar, nt * kGroupS * kChunk);
              // chunk j of the pair's first tile, then of the second, for kGroupS consecutive chunks
#pragma unroll
              for (int jj = 0; jj < kGroupS; ++jj) {
                const int j = kGroupS * g + jj;
                tma_load_3d(dst + jj * kDChunk, &tm_kv, bar, 64 * j, 0, blk0);
                if (nt == 2) tma_load_3d(dst + jj * kDChunk + kChunk, &tm_kv, bar, 64 * j, 0, blk1);
              }
            }
          }
        }
      }
      // every load issued has landed before the CTA may exit
      int dummy = 0;
      for (uint32_t i = 0; i < kSlots && i < c; ++i) {
        const uint32_t cl = c - 1 - i;
        mbar_wait<false>(smem_u32(&ctl.full[cl % kSlots]), (cl / kSlots) & 1, &dummy, drain_ns);
      }
      for (uint32_t i = sc_issued > 4 ? sc_issued - 4 : 0; kFp8 && i < sc_issued; ++i)
        mbar_wait<false>(smem_u32(&ctl.sc_full[i & 3]), (i >> 2) & 1, &dummy, drain_ns);
      if (!ok) set_status(a.status, MLA_ERR_TIMEOUT);
    }
  } else if (rank == 0 && warp == kMmaWarp) {
    // ------------------------------------------------------------------ score CTA: MMA issuer
    // The whole warp walks and waits, converged, and one elected lane issues (see elect_one): the score
    // MMAs are the kernel's critical path, and a single-lane branch computed and moved their operands one
    // by one (windows of 64 sequences x 65 tiles: 108 us, 101 us like this).
    const bool leader = elect_one();
    constexpr uint32_t idesc2 = idesc_bf16_f32(128, 128, false);   // a tile pair
    constexpr uint32_t idesc1 = idesc_bf16_f32(128, 64, false);    // a single tile
    constexpr uint32_t idesc2c = idesc_e4m3_f32(128, 128), idesc1c = idesc_e4m3_f32(128, 64);
    constexpr uint32_t idesc2l = idesc_f8_f32(128, 128, true, false), idesc1l = idesc_f8_f32(128, 64, true, false);   // lo
    // descriptor of ring slot 0's rows (K-major, 8-row groups 1 KB apart, the second tile right after the
    // first); 32 bytes along K add 2
    const uint64_t ring_desc = smem_desc(smem_u32(smem + kOffRingS), 16, 1024, kSwizzle128B);
    const uint64_t qr_desc = smem_desc(smem_u32(smem + kOffQr8), 16, 1024, kSwizzle128B);
    SegIter it(plan, a.seq_lens, a.B, tiles, cap, w, a.status);
    Segment sg;
    uint32_t slot = 0, phase = 0, u = 0, seg = 0;
    bool ok = true;
    while (ok && __any_sync(0xffffffffu, it.next(sg))) {
      const int tile_begin = __shfl_sync(0xffffffffu, sg.tile_begin, 0), tile_end = __shfl_sync(0xffffffffu, sg.tile_end, 0);
      ok = wait_warp(smem_u32(&ctl.q_full), seg & 1);
      if (!ok) break;
      tc_fence_after();
      for (int tile = tile_begin; ok && tile < tile_end; tile += 2, ++u) {
        const bool two = tile_end - tile >= 2;
        if (u >= 1) ok = wait_warp(smem_u32(&ctl.s_empty), (u & 1) ^ 1);
        if (!ok) break;
        tc_fence_after();
        // Loops around barrier waits stay rolled: unrolled, the pipelines of this kernel ran about
        // 1.4x slower on B200 (measured).
#pragma unroll 1
        for (int g = 0; g < (kFp8 ? kChunksS8 : kChunksS / kGroupS); ++g) {
          ok = wait_warp(smem_u32(&ctl.full[slot]), phase);
          if (!ok) break;
          tc_fence_after();
          const uint64_t bdesc = ring_desc + slot * (kSlotBytes >> 4);
          if (leader) {
            if constexpr (kFp8) {
              if (g < kChunksS8 - 1) {
                // 32 channels per step: eight TMEM columns of codes; hi, then lo into the same accumulator
                const uint32_t qa = tmem + kTmemQ + 32 * g, ic = two ? idesc2c : idesc1c, il = two ? idesc2l : idesc1l;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  mma_f8_ts(tmem + kTmemS8, qa + 8 * kk, bdesc + 2 * kk, ic, (g | kk) ? 1u : 0u);
                  mma_f8_ts(tmem + kTmemS8, qa + kTmemLo8 + 8 * kk, bdesc + 2 * kk, il, 1u);
                }
              } else {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  mma_ss(tmem + kTmemR8, qr_desc + 2 * kk, bdesc + 2 * kk, two ? idesc2 : idesc1, kk ? 1u : 0u);
              }
            } else {
              const uint32_t qa = tmem + kTmemQ + 8 * 4 * kGroupS * g;
#pragma unroll
              for (int jj = 0; jj < kGroupS; ++jj) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  // 16 channels per step: A = query words from TMEM, B = the pair's rows of chunk kGroupS g + jj
                  mma_ts(tmem + kTmemS, qa + 8 * (4 * jj + kk), bdesc + jj * (kDChunk >> 4) + 2 * kk, two ? idesc2 : idesc1,
                         (g | jj | kk) ? 1u : 0u);
                }
              }
            }
            mma_commit(smem_u32(&ctl.empty[slot]));   // the slot is free once these MMAs have read it
          }
          if (++slot == kSlots) {
            slot = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (leader) mma_commit(smem_u32(&ctl.s_full));
      }
      if (!ok) break;
      if (leader) mma_commit(smem_u32(&ctl.q_empty));
      ++seg;
    }
    int dummy = 0;
    if (leader) mma_commit(smem_u32(&ctl.drain));
    __syncwarp();
    mbar_wait<false>(smem_u32(&ctl.drain), 0, &dummy, drain_ns);
    if (!ok && lane == 0) set_status(a.status, MLA_ERR_TIMEOUT);
  } else if (rank == 0 && warp < kProducerWarp) {
    // ------------------------------------------------------------------ score CTA: softmax warps
    SegIter it(plan, a.seq_lens, a.B, tiles, cap, w, a.status);
    Segment sg;
    uint32_t t = 0, u = 0, seg = 0;   // tiles and pairs before this segment, segments
    bool ok = true;
    while (it.next(sg)) {
      const int n = sg.tile_end - sg.tile_begin;
      float m_run = -INFINITY, l_run = 0.f, l_tot = 0.f;   // l_run: this half's columns
      float m_top = -INFINITY, low_max = -INFINITY;        // e4m3 cache: highest reference; largest low pair
      int low = 0;                                         // ... and the number of low pairs under this reference
      bool poisoned = false;
      float scale_log2 = a.scale_log2;   // e4m3 cache: times 2^e, the power of two of this row's query
      if (ok) {
        // this segment's absorbed query into TMEM: of every row, half 0 loads the latent channels
        // [0, 256), half 1 the channels [256, 512) and the RoPE channels
        ok = wait_warp(smem_u32(&ctl.q_empty), (seg & 1) ^ 1);
        if (ok) {
          // in blocks of 128 bytes per row: eight lanes read a row's block side by side (instruction i:
          // row 8 (lane / 8) + i, piece lane % 8), then the pieces move to the row's own lane. Read one row per
          // lane (32 requests per load), a worker's first query took 8.5 us, like this 6.3.
          const int row0 = rg * kRows + 32 * quarter + (lane & ~7);   // query row of this lane group's first row
          const uint16_t* ql = (const uint16_t*)a.q_lat + ((size_t)sg.b * a.rows + row0) * kR + 256 * half + 8 * (lane & 7);
          const uint16_t* qr = (const uint16_t*)a.q_rope + ((size_t)sg.b * a.rows + row0) * kDR + 8 * (lane & 7);
          auto fetch = [&](int k, uint4 (&q)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              q[i] = row0 + i < a.rows
                         ? __ldg(reinterpret_cast<const uint4*>(k < 4 ? ql + (size_t)i * kR + 64 * k : qr + (size_t)i * kDR))
                         : make_uint4(0u, 0u, 0u, 0u);
          };
          // blocks in the order RoPE (k = 4; half 1 only), latent 0 .. 3, two of them on their way: block k is
          // number i0 = (k + 1) % 5
          uint4 n0[8], n1[8];
          auto start = [&] {
            if (half == 1) {
              fetch(4, n0);
              fetch(0, n1);
            } else {
              fetch(0, n0);
              fetch(1, n1);
            }
          };
          auto step = [&](int i0, uint4 (&q)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              q[i] = n0[i];
              n0[i] = n1[i];
            }
            if (i0 + 2 < 5) fetch(i0 + 1, n1);
          };
          auto words = [&](const uint4 (&q)[8], uint32_t (&w32)[32]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              w32[4 * i] = q[i].x;
              w32[4 * i + 1] = q[i].y;
              w32[4 * i + 2] = q[i].z;
              w32[4 * i + 3] = q[i].w;
            }
          };
          if constexpr (kFp8) {
            // The rows' largest magnitudes: over this half's channels (piece by piece of eight rows, then across
            // the eight lanes that share them), then with the other half's.
            float mx[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) mx[i] = 0.f;
            {
              uint4 q[4][8];
#pragma unroll
              for (int k = 0; k < 4; ++k) fetch(k, q[k]);
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  mx[i] = fmaxf(mx[i], fmaxf(fmaxf(bf16x2_amax(q[k][i].x), bf16x2_amax(q[k][i].y)),
                                             fmaxf(bf16x2_amax(q[k][i].z), bf16x2_amax(q[k][i].w))));
            }
            start();
            if (half == 1) {   // (the RoPE part as 2^-64 of itself: bf16 keeps its bits under any e, as long as sums stay finite)
#pragma unroll
              for (int i = 0; i < 8; ++i)
                mx[i] = fmaxf(mx[i], 0x1p-64f * fmaxf(fmaxf(bf16x2_amax(n0[i].x), bf16x2_amax(n0[i].y)),
                                                     fmaxf(bf16x2_amax(n0[i].z), bf16x2_amax(n0[i].w))));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int o = 1; o < 8; o *= 2) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
            float m = mx[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) m = (lane & 7) == i ? mx[i] : m;   // row 8 (lane / 8) + lane % 8: this lane's
            float* qmax = reinterpret_cast<float*>(smem + kOffQmax8);
            qmax[half * kRows + row] = m;
            warp_arrive(smem_u32(&ctl.qbar[quarter]));
            ok = wait_warp(smem_u32(&ctl.qbar[quarter]), seg & 1);
            const int e = split_exponent(fmaxf(m, qmax[(half ^ 1) * kRows + row]));
            const float down = __uint_as_float((uint32_t)(127 - e) << 23);
            scale_log2 = a.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll 1
            for (int i0 = half ? 0 : 1; i0 < 5; ++i0) {
              const int k = (i0 + 4) % 5;
              uint4 q[8];
              uint32_t w32[32];
              step(i0, q);
              transpose_pieces<8>(q);
              words(q, w32);
              if (k < 4) {   // 64 channels as 16 words of hi codes and 16 of lo
                uint32_t hl[32];
#pragma unroll
                for (int i = 0; i < 16; ++i) split_f8(w32[2 * i], w32[2 * i + 1], down, hl[i], hl[16 + i]);
                tmem_st16(tmem + lane_off + kTmemQ + 64 * half + 16 * k, hl);
                tmem_st16(tmem + lane_off + kTmemQ + kTmemLo8 + 64 * half + 16 * k, hl + 16);
              } else {       // RoPE channels, scaled alike: 128 bytes of the K-major operand, 128-byte swizzle
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  w32[i] = pack_bf16x2(__uint_as_float(w32[i] << 16) * down, __uint_as_float(w32[i] & 0xFFFF0000u) * down);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  *reinterpret_cast<uint4*>(smem + kOffQr8 + row * 128 + ((i ^ (row & 7)) << 4)) =
                      make_uint4(w32[4 * i], w32[4 * i + 1], w32[4 * i + 2], w32[4 * i + 3]);
                fence_proxy_async_smem();
              }
            }
          } else {
            start();
#pragma unroll 1   // rolled: code that runs once per segment waits for its instructions
            for (int i0 = half ? 0 : 1; i0 < 5; ++i0) {
              const int k = (i0 + 4) % 5;
              uint4 q[8];
              uint32_t w32[32];
              step(i0, q);
              transpose_pieces<8>(q);
              words(q, w32);
              // column = word index of the absorbed query row
              tmem_st32(tmem + lane_off + kTmemQ + (k < 4 ? 128 * half + 32 * k : 256), w32);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          warp_arrive(smem_u32(&ctl.q_full));
        }
        // (here, while the first pair is scored: its loads would hold the next segment up)
        poisoned = segment_poisoned(a, tiles, sg.b, sg.tile_begin, sg.tile_end);
        int n_row = valid_row ? (a.causal ? sg.Lc - a.Sq + 1 + s_idx : sg.Lc) : 0;
        if (n_row < 0) n_row = 0;
        for (int li = 0; ok && li < n; li += 2, ++u) {
          const int nt = min(2, n - li);            // tiles in this pair
          const bool mine = half < nt;              // this half has a tile
          const int tile = sg.tile_begin + li + half;
          const bool last_pair = li + 2 >= n;
          ok = wait_warp(smem_u32(&ctl.s_full), u & 1);
          if (!ok) break;
          tc_fence_after();
          uint32_t v[64];
          constexpr uint32_t kScores = kFp8 ? kTmemS8 : kTmemS;
          tmem_ld32(tmem + lane_off + kScores + 64 * half, v);
          tmem_ld32(tmem + lane_off + kScores + 64 * half + 32, v + 32);
          uint32_t r[kFp8 ? 64 : 1];   // e4m3 cache: the RoPE scores
          if constexpr (kFp8) {
            tmem_ld32(tmem + lane_off + kTmemR8 + 64 * half, r);
            tmem_ld32(tmem + lane_off + kTmemR8 + 64 * half + 32, r + 32);
          }
          tmem_wait_ld();
          tc_fence_before();
          warp_arrive(smem_u32(&ctl.s_empty));
          // e4m3 cache: the tile's token scales, and this warp's copy of their logarithms and of themselves
          const float* sc = reinterpret_cast<const float*>(smem + kOffScale8) + (u & 3) * 128 + 64 * half;
          float* lsc = reinterpret_cast<float*>(smem + kOffLog8) + warp * 128;
          if constexpr (kFp8) {
            ok = wait_warp(smem_u32(&ctl.sc_full[u & 3]), (u >> 2) & 1);
            if (!ok) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float s = sc[lane + 32 * h];
              lsc[lane + 32 * h] = __log2f(fmaxf(s, kScaleFloor));
              // (behind p = 0 of a token that is not seen, whose scale may be anything)
              lsc[64 + lane + 32 * h] = fabsf(s) < INFINITY ? s : 0.f;
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 64; j += 4) {
              const ulonglong2 s4 = *reinterpret_cast<const ulonglong2*>(sc + j);
#pragma unroll
              for (int i = 0; i < 4; i += 2) {
                const unsigned long long x =
                    fma2(f2_pack(__uint_as_float(v[j + i]), __uint_as_float(v[j + i + 1])), i ? s4.y : s4.x,
                         f2_pack(__uint_as_float(r[j + i]), __uint_as_float(r[j + i + 1])));
                float x0, x1;
                f2_unpack(x, x0, x1);
                v[j + i] = __float_as_uint(x0);
                v[j + i + 1] = __float_as_uint(x1);
              }
            }
          }
          // The pair's row maximum of the scaled scores (log2 units) from both halves. A full tile
          // keeps the raw scores and takes the extreme with three-input min / max (the scale folds
          // into the exponent's FMA below); a partial one masks the columns past the row's
          // attended tokens after scaling.
          const int valid = mine ? min(max(n_row - tile * kBS, 0), kBS) : 0;
          const WindowCols cols(a, mine ? n_row : 0, kWindow ? tiles.block(tile, sg.Lc) * kBS : 0, kBS);
          const bool full = kWindow ? cols.all(kBS) : valid == kBS;
          float mh;
          if (kFp8) {   // the maximum of score + log2 of the token's scale
            mh = -INFINITY;
            const float c = full ? scale_log2 : 1.f;
            if (!full) {
#pragma unroll
              for (int j = 0; j < 64; ++j)
                v[j] = __float_as_uint(cols.sees(j) ? __uint_as_float(v[j]) * scale_log2 : -INFINITY);
            }
            const unsigned long long c2 = f2_pack(c, c);
#pragma unroll
            for (int j = 0; j < 64; j += 4) {
              const ulonglong2 l4 = *reinterpret_cast<const ulonglong2*>(lsc + j);
#pragma unroll
              for (int i = 0; i < 4; i += 2) {
                float t0, t1;
                f2_unpack(fma2(f2_pack(__uint_as_float(v[j + i]), __uint_as_float(v[j + i + 1])), c2, i ? l4.y : l4.x), t0, t1);
                mh = max3f(mh, t0, t1);
              }
            }
          } else if (full) {
            float r = __uint_as_float(v[0]);
            if (scale_log2 >= 0.f) {
#pragma unroll
              for (int j = 1; j < 63; j += 2) r = max3f(r, __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
              r = fmaxf(r, __uint_as_float(v[63]));
            } else {
#pragma unroll
              for (int j = 1; j < 63; j += 2) r = min3f(r, __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
              r = fminf(r, __uint_as_float(v[63]));
            }
            mh = r * scale_log2;
          } else {
            mh = -INFINITY;
#pragma unroll
            for (int j = 0; j < 64; ++j) {
              const bool see = kWindow ? cols.sees(j) : j < valid;
              const float x = see ? __uint_as_float(v[j]) * scale_log2 : -INFINITY;
              v[j] = __float_as_uint(x);
              mh = fmaxf(mh, x);
            }
          }
          ctl.xmax[u & 1][half][row] = mh;
          warp_arrive(smem_u32(&ctl.xbar[quarter]));
          ok = wait_warp(smem_u32(&ctl.xbar[quarter]), u & 1);   // bounded: the partner warp may have aborted
          if (!ok) break;
          const float mt = fmaxf(mh, ctl.xmax[u & 1][half ^ 1][row]);
          bool move = mt > m_run + kRescaleThreshold;   // the reference moves
          float m_new = kFp8 ? mt - kHeadroom8 : mt;
          if constexpr (kFp8) {
            const bool is_low = mt < m_run + kLow8 && mt > -INFINITY && m_run > m_top - kDepth8;
            if (move) m_top = fmaxf(m_top, m_new);
            if (is_low) {
              ++low;
              low_max = fmaxf(low_max, mt);
            }
            // one row's turn lowers those of the warp whose pair is low too (both halves decide alike)
            if (__any_sync(0xffffffffu, low >= kLowPairs8) && is_low) {
              move = true;
              m_new = fmaxf(low_max - kHeadroom8, m_top - kDepth8);
            }
            if (move) {
              low = 0;
              low_max = -INFINITY;
            }
          }
          const float alpha = (move && m_run != -INFINITY) ? ex2_approx(m_run - m_new) : 1.f;
          if (move) {
            l_run *= alpha;
            m_run = m_new;
          }
          uint32_t pk[32];
          float psum = 0.f;
          if (m_run != -INFINITY) {
            // p = 2^(c s - m) two columns at a time: c = the scale (full tile) or 1 (scaled, masked)
            const float c = full ? scale_log2 : 1.f;
            const unsigned long long cc = f2_pack(c, c), nm = f2_pack(-m_run, -m_run);
            unsigned long long acc = f2_pack(0.f, 0.f);
            if constexpr (kFp8) {
              // four columns at a time: p, its sum, and p s_t as one word of hi and one of lo codes
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const ulonglong2 s4 = *reinterpret_cast<const ulonglong2*>(lsc + 64 + 4 * k);
                uint32_t hi[2], lo[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const int j = 4 * k + 2 * h;
                  float x0, x1;
                  f2_unpack(fma2(f2_pack(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), cc, nm), x0, x1);
                  const unsigned long long p2 = f2_pack(ex2_approx(x0), ex2_approx(x1));
                  acc = add2(acc, p2);
                  two_terms(mul2(p2, h ? s4.y : s4.x), hi[h], lo[h]);
                }
                pk[k] = hi[0] | (hi[1] << 16);
                pk[16 + k] = lo[0] | (lo[1] << 16);
              }
            }
#pragma unroll
            for (int k = 0; k < (kFp8 ? 0 : 32); ++k) {
              float x0, x1;
              f2_unpack(fma2(f2_pack(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), cc, nm), x0, x1);
              const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
              acc = add2(acc, f2_pack(p0, p1));
              pk[k] = pack_bf16x2(p0, p1);
            }
            float s0, s1;
            f2_unpack(acc, s0, s1);
            psum = s0 + s1;
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) pk[k] = 0u;
          }
          l_run += psum;
          if (last_pair) {
            // the segment's row sum over both halves, for the output CTA's normalisation
            ctl.xsum[half][row] = l_run;
            warp_arrive(smem_u32(&ctl.sbar[quarter]));
            ok = wait_warp(smem_u32(&ctl.sbar[quarter]), seg & 1);
            if (!ok) break;
            l_tot = l_run + ctl.xsum[half ^ 1][row];
          }
          if (mine) {
            const bool last_tile = last_pair && half == nt - 1;
            const float invl = (last_tile && l_tot > 0.f) ? 1.f / l_tot : 0.f;
            // O is rescaled before the pair's first tile only
            const float fac = half == 0 ? alpha : 1.f;
            // outgoing buffer tt % kStage is free once tile tt - kStage has reached the output CTA
            const uint32_t tt = t + li + half, sb = tt % kStage;
            bool free_buf = true;
            if (lane == 0 && tt >= (uint32_t)kStage)
              free_buf = mbar_wait<true>(smem_u32(&ctl.sent[sb]), ((tt / kStage) & 1) ^ 1, abort, timeout_ns);
            ok = __shfl_sync(0xffffffffu, free_buf, 0);
            if (!ok) break;
            // this row of the tile's message: P as [8-token chunk][row][8 tokens] (8-row x 16-byte
            // core matrices, the K-major layout the output CTA's PV reads), then the row's
            // (rescale factor, 1 / row sum)
            uint8_t* msg = smem + kOffMsg + sb * kMsgBytes;
#pragma unroll
            for (int cc = 0; cc < 8; ++cc)
              *reinterpret_cast<uint4*>(msg + cc * (kRows * 16) + row * 16) =
                  make_uint4(pk[4 * cc], pk[4 * cc + 1], pk[4 * cc + 2], pk[4 * cc + 3]);
            *reinterpret_cast<float2*>(msg + kPBytes + row * 8) = make_float2(fac, invl);
            fence_proxy_async_smem();   // for the bulk copy that sends the buffer
            warp_arrive(smem_u32(&ctl.written[sb]));
          }
        }
        t += n;
        ++seg;
      }
      // log-sum-exp of the rows of this segment (the output CTA writes the values)
      if (valid_row && half == 0) {
        float lse_v = l_tot > 0.f ? (m_run + log2f(l_tot)) * 0.69314718055994531f : -INFINITY;
        if (!ok || poisoned) lse_v = __uint_as_float(0x7FC00000u);
        if (sg.splits == 1)
          a.lse[(size_t)sg.b * a.rows + grow] = lse_v;
        else
          a.lse_part[(size_t)(w + sg.b) * a.rows + grow] = lse_v;
      }
    }
    if (!ok) set_status(a.status, MLA_ERR_TIMEOUT);
  } else if (rank == 0 && warp == kPostWarp) {
    // ------------------------------------------------------------------ score CTA: message sends
    // In tile order: once the 128 softmax threads of a tile have written its message and the
    // PV that last read receive buffer t % kRxBufs has completed, one bulk copy moves the
    // message into the output CTA's shared memory (bytes complete on its barrier).
    if (lane == 0) {
      SegIter it(plan, a.seq_lens, a.B, tiles, cap, w, a.status);
      Segment sg;
      uint32_t t = 0;
      bool ok = true;
      while (ok && it.next(sg)) {
        for (int li = sg.tile_begin; li < sg.tile_end; ++li, ++t) {
          const uint32_t sb = t % kStage, rb = t % kRxBufs;
          ok = mbar_wait<false>(smem_u32(&ctl.written[sb]), (t / kStage) & 1, abort, timeout_ns);
          if (ok && t >= (uint32_t)kRxBufs)
            ok = mbar_wait<true>(smem_u32(&ctl.credit[rb]), ((t / kRxBufs) & 1) ^ 1, abort, timeout_ns);
          if (!ok) break;
          bulk_copy_to_peer(mapa(smem_u32(smem + kOffRx + rb * kMsgBytes), peer),
                            smem_u32(smem + kOffMsg + sb * kMsgBytes), kMsgBytes,
                            mapa(smem_u32(&ctl.rx_full[rb]), peer));
        }
      }
      // the PV completions of the last tiles still signal our credit barriers: wait for them
      // (bounded) so that no arrival can reach this CTA's shared memory after it exits
      int dummy = 0;
      for (uint32_t i = 0; i < (uint32_t)kRxBufs && i < t; ++i) {
        const uint32_t tl = t - 1 - i;
        mbar_wait<true>(smem_u32(&ctl.credit[tl % kRxBufs]), (tl / kRxBufs) & 1, &dummy, drain_ns);
      }
      if (!ok) set_status(a.status, MLA_ERR_TIMEOUT);
    }
  } else if (kSparse && warp == kProducerWarp) {
    // ------------------------------------------------------------------ output CTA: row gathers
    // lanes 0-15 fetch the tile's rows 4L .. 4L + 3, each half stage's four 64-channel chunks
    // with one 4-row gather each (the layout of the tiled 4-D box)
    SegIter it(plan, a.seq_lens, a.B, tiles, cap, w, a.status);
    Segment sg;
    uint32_t h = 0;
    bool ok = true;
    while (ok && it.next(sg)) {
      for (int tile = sg.tile_begin; ok && tile < sg.tile_end; ++tile) {
        const bool act = lane < 16;
        int r4[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) r4[m] = act ? sparse_row(a, sg.b, tile * kBS + 4 * lane + m, sg.Lc) : 0;
#pragma unroll 1   // rolled: see the score MMA loop
        for (int hc = 0; hc < 2; ++hc, ++h) {
          const uint32_t hs = h % kHalves;
          bool free_half = true;
          if (lane == 0 && h >= (uint32_t)kHalves)
            free_half = mbar_wait<false>(smem_u32(&ctl.oempty[hs]), ((h / kHalves) & 1) ^ 1, abort, timeout_ns);
          ok = __shfl_sync(0xffffffffu, free_half, 0);
          if (!ok) break;
          const uint32_t bar = smem_u32(&ctl.ofull[hs]);
          const uint32_t base = smem_u32(smem + kOffRingO + hs * kHalfBytes);
          if (lane == 0) mbar_arrive_expect_tx(bar, kHalfBytes);
          __syncwarp();
          if (act) {
#pragma unroll
            for (int cc = 0; cc < 4; ++cc)
              tma_gather4(base + cc * kChunk + lane * 512, &tm_kv, bar, 256 * hc + 64 * cc, r4);
          }
        }
      }
    }
    if (lane == 0) {
      int dummy = 0;
      for (uint32_t i = 0; i < kHalves && i < h; ++i) {
        const uint32_t hl = h - 1 - i;
        mbar_wait<false>(smem_u32(&ctl.ofull[hl % kHalves]), (hl / kHalves) & 1, &dummy, drain_ns);
      }
      if (!ok) set_status(a.status, MLA_ERR_TIMEOUT);
    }
  } else if (warp == kProducerWarp) {
    // ------------------------------------------------------------------ output CTA: TMA producer
    if (lane == 0) {
      SegIter it(plan, a.seq_lens, a.B, tiles, cap, w, a.status);
      Segment sg;
      uint32_t h = 0;
      bool ok = true;
      while (ok && it.next(sg)) {
        for (int tile = sg.tile_begin; ok && tile < sg.tile_end; ++tile) {
          const int blk = tile_block(a, sg.b, tiles.block(tile, sg.Lc));
#pragma unroll 1   // rolled: see the score MMA loop
          for (int hc = 0; hc < 2; ++hc, ++h) {
            const uint32_t hs = h % kHalves;
            if (h >= (uint32_t)kHalves &&
                !mbar_wait<false>(smem_u32(&ctl.oempty[hs]), ((h / kHalves) & 1) ^ 1, abort, timeout_ns)) {
              ok = false;
              break;
            }
            const uint32_t bar = smem_u32(&ctl.ofull[hs]);
            const uint32_t base = smem_u32(smem + kOffRingO + hs * kHalfBytes);
            mbar_arrive_expect_tx(bar, kHalfBytes);
            tma_load_4d(base, &tm_kv4, bar, 0, 0, (kFp8 ? 2 : 4) * hc, blk);   // latent chunks of 256 channels
          }
        }
      }
      int dummy = 0;
      for (uint32_t i = 0; i < kHalves && i < h; ++i) {
        const uint32_t hl = h - 1 - i;
        mbar_wait<false>(smem_u32(&ctl.ofull[hl % kHalves]), (hl / kHalves) & 1, &dummy, drain_ns);
      }
      if (!ok) set_status(a.status, MLA_ERR_TIMEOUT);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ output CTA: MMA issuer (converged warp)
    const bool leader = elect_one();
    constexpr uint32_t idesc_pv = kFp8 ? idesc_e4m3_f32(128, 256, true) : idesc_bf16_f32(128, 256, true);
    constexpr uint32_t idesc_lo = idesc_f8_f32(128, 256, true, false, true);   // e4m3 cache: P's lo terms are e5m2
    // A = P[128 rows][16 tokens per step] (K-major); the message's P: 8-row x 16-byte core matrices, 128
    // bytes apart along the rows, 2 KB apart along the tokens
    const uint64_t rx_desc = smem_desc(smem_u32(smem + kOffRx), 2048, 128, kSwizzleNone);
    // B = C[16 tokens][256 channels], channels contiguous: 64-channel chunks 8 KB apart, 8-token groups 1 KB
    // apart. e4m3 cache: steps of 32 tokens, the hi terms of P (chunks of 16 tokens 0-3 of the message) in
    // the first two and the lo terms (4-7) in the others; 128-channel chunks
    const uint64_t ring_desc = smem_desc(smem_u32(smem + kOffRingO), kChunk, 1024, kSwizzle128B);
    SegIter it(plan, a.seq_lens, a.B, tiles, cap, w, a.status);
    Segment sg;
    uint32_t rb = 0, rx_phase = 0, hs = 0, phase = 0;
    bool ok = true;
    while (ok && __any_sync(0xffffffffu, it.next(sg))) {
      const int n = __shfl_sync(0xffffffffu, sg.tile_end - sg.tile_begin, 0);
      for (int li = 0; li < n; ++li) {
        ok = wait_warp(smem_u32(&ctl.p_ready[rb]), rx_phase);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1   // rolled: see the score MMA loop
        for (int hc = 0; hc < 2; ++hc) {
          ok = wait_warp(smem_u32(&ctl.ofull[hs]), phase);
          if (!ok) break;
          tc_fence_after();
          const uint64_t adesc = rx_desc + rb * (kMsgBytes >> 4), bdesc = ring_desc + hs * (kHalfBytes >> 4);
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint32_t acc = (li > 0 || kk > 0) ? 1u : 0u;
              if constexpr (kFp8)
                mma_f8_ss(tmem + 256 * hc, adesc + kk * (4096 >> 4), bdesc + (kk & 1) * (4096 >> 4), kk < 2 ? idesc_pv : idesc_lo,
                          acc);
              else
                mma_ss(tmem + 256 * hc, adesc + kk * (4096 >> 4), bdesc + kk * (2048 >> 4), idesc_pv, acc);
            }
            mma_commit(smem_u32(&ctl.oempty[hs]));
          }
          if (++hs == kHalves) {
            hs = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (leader) {
          mma_commit(smem_u32(&ctl.pv_done[rb]));   // O is free again after this PV
          // the receive buffer goes back to the score CTA when this PV has completed
          mma_commit_to_ctas(smem_u32(&ctl.credit[rb]), (uint16_t)(1u << peer));
        }
        if (++rb == kRxBufs) {
          rb = 0;
          rx_phase ^= 1;
        }
      }
    }
    int dummy = 0;
    if (leader) mma_commit(smem_u32(&ctl.drain));
    __syncwarp();
    mbar_wait<false>(smem_u32(&ctl.drain), 0, &dummy, drain_ns);
    if (!ok && lane == 0) set_status(a.status, MLA_ERR_TIMEOUT);
  } else if (warp < kProducerWarp) {
    // ------------------------------------------------------------------ output CTA: row warps
    // thread = row; warp q works on O columns [0, 256) of its rows, warp q + 4 on [256, 512)
    const uint32_t rx = smem_u32(smem + kOffRx);
    const uint32_t col0 = 256 * half;
    SegIter it(plan, a.seq_lens, a.B, tiles, cap, w, a.status);
    Segment sg;
    uint32_t t = 0;
    bool ok = true;
    while (it.next(sg)) {
      const int n = sg.tile_end - sg.tile_begin;
      float inv_l = 0.f;
      const bool poisoned = segment_poisoned(a, tiles, sg.b, sg.tile_begin, sg.tile_end);   // before the first message
      if (ok) {
        const int last_tile = tiles.count(sg.Lc) - 1;
        const int tail = sg.Lc % kBS;
        for (int li = 0; li < n; ++li, ++t) {
          const uint32_t rb = t % kRxBufs, sb = t % kStage;
          const int tile = sg.tile_begin + li;
          ok = wait_warp(smem_u32(&ctl.rx_full[rb]), (t / kRxBufs) & 1);
          if (!ok) break;
          if (threadIdx.x == 0) {
            // re-arm for tile t + kRxBufs (its bytes can only come after this tile's PV), and hand
            // the score CTA's outgoing buffer of this tile back (the copy has read it)
            mbar_arrive_expect_tx(smem_u32(&ctl.rx_full[rb]), kMsgBytes);
            mbar_arrive_remote_relaxed(mapa(smem_u32(&ctl.sent[sb]), peer));
          }
          float2 fl;
          asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                       : "=f"(fl.x), "=f"(fl.y)
                       : "r"(rx + rb * kMsgBytes + kPBytes + (uint32_t)row * 8));
          const float alpha = fl.x;
          if (li == n - 1) inv_l = fl.y;
          if (li >= 1 && __any_sync(0xffffffffu, alpha != 1.f)) {
            // O holds the tiles before t: wait for their PV, then scale this row's half
            const uint32_t tp = t - 1;
            ok = wait_warp(smem_u32(&ctl.pv_done[tp % kRxBufs]), (tp / kRxBufs) & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < 8; ++cc) {
              uint32_t v[32];
              tmem_ld32(tmem + lane_off + col0 + 32 * cc, v);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
              tmem_st32(tmem + lane_off + col0 + 32 * cc, v);
            }
            tmem_wait_st();
          }
          if constexpr (kWindow) {
            // Tokens that no row sees may hold anything (NaN) as well: cache slots past the
            // sequence end, and those of a boundary block between the sinks and the earliest
            // window. The tile keeps columns [0, sink) and [first, end).
            const int base = tiles.block(tile, sg.Lc) * kBS;
            const int sink = min(max(min(a.sinks, sg.Lc) - base, 0), kBS);
            const int first = max(min(max(tiles.lo(sg.Lc) - base, 0), kBS), sink), end = min(sg.Lc - base, kBS);
            if (sink < first || end < kBS) {
              const uint32_t h0 = 2 * t, h1 = 2 * t + 1;
              ok = wait_warp(smem_u32(&ctl.ofull[h0 % kHalves]), (h0 / kHalves) & 1) &&
                   wait_warp(smem_u32(&ctl.ofull[h1 % kHalves]), (h1 / kHalves) & 1);
              if (!ok) break;
              const int from = min(first, end);   // rows to zero: [sink, from) and [end, 64)
              const int hole = from - sink, gone = hole + (kBS - end);
              constexpr int kCk = kFp8 ? 4 : 8;   // 128-byte chunks of a token's row
              for (int i = threadIdx.x; i < 8 * kCk * gone; i += kRowThreads) {
                const int ck = i % kCk, pc = (i / kCk) & 7, k = i / (8 * kCk);
                const int tok = k < hole ? sink + k : end + (k - hole);
                const uint32_t hs = (ck < kCk / 2 ? h0 : h1) % kHalves;
                *reinterpret_cast<uint4*>(smem + kOffRingO + hs * kHalfBytes + (ck % (kCk / 2)) * kChunk + tok * 128 + pc * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
              }
              fence_proxy_async_smem();
            }
          } else if (tile == last_tile && tail != 0) {
            // cache slots past the sequence end may hold anything (NaN): zero those token rows
            // of both half stages before the PV reads them (P is 0 there, but 0 * NaN is not)
            const uint32_t h0 = 2 * t, h1 = 2 * t + 1;
            ok = wait_warp(smem_u32(&ctl.ofull[h0 % kHalves]), (h0 / kHalves) & 1) &&
                 wait_warp(smem_u32(&ctl.ofull[h1 % kHalves]), (h1 / kHalves) & 1);
            if (!ok) break;
            const int per_chunk = (kBS - tail) * 8;   // 16-byte pieces per chunk
            for (int i = threadIdx.x; i < 8 * per_chunk; i += kRowThreads) {
              const int ck = i / per_chunk, rem = i % per_chunk;
              const uint32_t hs = (ck < 4 ? h0 : h1) % kHalves;
              uint8_t* p = smem + kOffRingO + hs * kHalfBytes + (ck & 3) * kChunk + (tail + rem / 8) * 128 + (rem % 8) * 16;
              *reinterpret_cast<uint4*>(p) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
          tc_fence_before();
          warp_arrive(smem_u32(&ctl.p_ready[rb]));
        }
        if (ok) ok = wait_warp(smem_u32(&ctl.pv_done[(t - 1) % kRxBufs]), ((t - 1) / kRxBufs) & 1);
      }
      // epilogue: O / l -> out (single split) or the normalised partial (several splits)
      const bool nan_rows = !ok || poisoned;
      const bool direct = sg.splits == 1;
      if (ok) tc_fence_after();
      // Eight lanes write 128 bytes of a row side by side (transpose_pieces): the row of instruction i is
      // the group's i-th. One row per lane took 11.5 us for 128 x 512 fp32 (LSU requests), this 5.5.
      const int row0 = rg * kRows + 32 * quarter + (lane & ~7);
      const size_t qrow0 = (size_t)sg.b * a.rows + row0, prow0 = (size_t)(w + sg.b) * a.rows + row0;
      const bool bf16_out = direct && a.out_dtype == kBF16;
      auto load32 = [&](int cc, float* f) {
        uint32_t v[32];
        if (ok) {
          tmem_ld32(tmem + lane_off + col0 + 32 * cc, v);
          tmem_wait_ld();
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) f[i] = nan_rows ? __uint_as_float(0x7FC00000u) : __uint_as_float(v[i]) * inv_l;
      };
      if (bf16_out) {
#pragma unroll 1
        for (int cc = 0; cc < 8; cc += 2) {
          uint4 u[8];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float f[32];
            load32(cc + h, f);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              u[4 * h + i] = make_uint4(pack_bf16x2(f[8 * i], f[8 * i + 1]), pack_bf16x2(f[8 * i + 2], f[8 * i + 3]),
                                        pack_bf16x2(f[8 * i + 4], f[8 * i + 5]), pack_bf16x2(f[8 * i + 6], f[8 * i + 7]));
          }
          transpose_pieces<8>(u);
          uint16_t* dst = (uint16_t*)a.out + qrow0 * kR + col0 + 32 * cc + 8 * (lane & 7);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (row0 + i < a.rows) *reinterpret_cast<uint4*>(dst + (size_t)i * kR) = u[i];
        }
      } else {
        float* base = direct ? (float*)a.out + qrow0 * kR : a.o_part + prow0 * kR;
#pragma unroll 1
        for (int cc = 0; cc < 8; ++cc) {
          float f[32];
          load32(cc, f);
          uint4 u[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            u[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                              __float_as_uint(f[4 * i + 3]));
          transpose_pieces<8>(u);
          float* dst = base + col0 + 32 * cc + 4 * (lane & 7);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (row0 + i < a.rows) *reinterpret_cast<uint4*>(dst + (size_t)i * kR) = u[i];
        }
      }
      tc_fence_before();
    }
    if (!ok) set_status(a.status, MLA_ERR_TIMEOUT);
  }

  // ------------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  cluster_sync();   // no CTA leaves while its peer may still write its shared memory
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

}  // namespace

cudaError_t launch_pair_decode(const DecodeArgs& a, cudaStream_t s) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return cudaErrorInvalidValue;
  const bool sparse = a.sel_idx != nullptr;
  if (sparse && (a.Sq != 1 || a.causal)) return cudaErrorInvalidValue;
  const bool windowed = a.window > 0, fp8 = a.cache_dtype == kE4M3;
  if (sparse && windowed) return cudaErrorInvalidValue;
  if (fp8 && !windowed) return cudaErrorInvalidValue;
  CUtensorMap tm, tm4, tmr, tms;
  auto encode = [&](CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims,
                    const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(m, type, rank, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (fp8) {
    const cuuint64_t nb = (cuuint64_t)a.num_blocks;
    // codes [num_blocks][64][512], boxes of 128 channels x 64 tokens; the same as (128 channels, 64
    // tokens, 4 chunks, blocks), boxes of two chunks; RoPE keys [num_blocks][64][64] bf16; scales
    const cuuint64_t d3[3] = {kR, kBS, nb}, s3[2] = {kR, (cuuint64_t)kBS * kR};
    const cuuint64_t d4[4] = {128, kBS, kR / 128, nb}, s4[3] = {kR, 128, (cuuint64_t)kBS * kR};
    const cuuint64_t dr[3] = {kDR, kBS, nb}, sr[2] = {kDR * 2, (cuuint64_t)kBS * kDR * 2};
    const cuuint64_t ds[3] = {kBS, 1, nb}, ss[2] = {kBS * 4, kBS * 4};
    const cuuint32_t b3[3] = {128, kBS, 1}, b4[4] = {128, kBS, 2, 1}, br[3] = {kDR, kBS, 1}, bs[3] = {kBS, 1, 1};
    if (!encode(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.cache, d3, s3, b3, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode(&tm4, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, a.cache, d4, s4, b4, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode(&tmr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.k_rope, dr, sr, br, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode(&tms, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, a.kv_scale, ds, ss, bs, CU_TENSOR_MAP_SWIZZLE_NONE))
      return cudaErrorInvalidValue;
  } else if (sparse) {
    // the cache as rows [num_blocks * 64][576] bf16: one-row boxes of 64 channels (128 bytes,
    // 128-byte swizzle) for 4-row gathers; rows past the cache read as zeros
    const cuuint64_t dims[2] = {(cuuint64_t)(kR + kDR), (cuuint64_t)a.num_blocks * kBS};
    const cuuint64_t strides[1] = {(cuuint64_t)(kR + kDR) * 2};
    const cuuint32_t box[2] = {64, 1};
    const cuuint32_t estr[2] = {1, 1};
    if (fn(&tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(a.cache), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
    tm4 = tm;   // unused by the gathering producers
  } else {
    // the cache [num_blocks][64][576] bf16, boxes of 64 channels x 64 tokens, 128-byte swizzle
    const cuuint64_t dims[3] = {(cuuint64_t)(kR + kDR), (cuuint64_t)kBS, (cuuint64_t)a.num_blocks};
    const cuuint64_t strides[2] = {(cuuint64_t)(kR + kDR) * 2, (cuuint64_t)kBS * (kR + kDR) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)kBS, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    if (fn(&tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.cache), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
    // the same cache as (64 channels, 64 tokens, 9 channel chunks, blocks): one box = 4 chunks of
    // a block, written as [chunk][token][128 bytes], the layout of four 3-D boxes side by side
    const cuuint64_t dims4[4] = {64, (cuuint64_t)kBS, (cuuint64_t)(kR + kDR) / 64, (cuuint64_t)a.num_blocks};
    const cuuint64_t strides4[3] = {(cuuint64_t)(kR + kDR) * 2, 128, (cuuint64_t)kBS * (kR + kDR) * 2};
    const cuuint32_t box4[4] = {64, (cuuint32_t)kBS, 4, 1};
    const cuuint32_t estr4[4] = {1, 1, 1, 1};
    if (fn(&tm4, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a.cache), dims4, strides4, box4, estr4,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  if (!fp8) tmr = tms = tm;   // unused by the bf16 kernels
  auto kernel = sparse     ? pair_decode_kernel<true, false, false>
                : fp8      ? pair_decode_kernel<false, true, true>
                : windowed ? pair_decode_kernel<false, true, false>
                           : pair_decode_kernel<false, false, false>;
  const int smem = fp8 ? kSmemBytes8 : kSmemBytes;
  static std::once_flag attr_once[4][64];
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t attr_err = cudaSuccess;
  std::call_once(attr_once[sparse ? 1 : fp8 ? 3 : windowed ? 2 : 0][dev & 63],
                 [&] { attr_err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
  if (attr_err != cudaSuccess) return attr_err;
  const int n_rg = (a.rows + kRows - 1) / kRows;
  const dim3 grid(2 * a.W * n_rg);
  kernel<<<grid, kThreads, smem, s>>>(tm, tm4, tmr, tms, a, n_rg, wait_timeout_ns(), drain_timeout_ns());
  return cudaGetLastError();
}

}  // namespace mla
