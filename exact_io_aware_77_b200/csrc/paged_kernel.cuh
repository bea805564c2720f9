// Attention of a few new query rows per sequence over a paged key/value cache.
//
// Sequence b holds lengths[b] keys (read on the device, so that a captured graph follows a
// growing cache); key j lies in row j % page_size of page table[b][j / page_size].  Of its N_q query
// rows the first counts[b] are new ones (all, without counts): row i stands at position
// lengths[b] - counts[b] + i, where the causal and window masks apply.  Rows past the count, which are
// padding, and rows without an allowed key (an idle slot of the batch has length 0) give O = 0 and
// L = -inf.
//
// One item is one (sequence, K/V head, block of 16 of the head's group * N_q rows); its work is
// the sequence's steps of 16, 32 or 64 keys.  As lengths differ, the items' steps are laid end to
// end on one line, a small surcharge standing before each item for its set-up, and the line is cut
// into pieces (PgCut) that single warps work through: a long sequence spreads over as many warps as
// it needs, and the partial results number two per piece at most (the items that it shares with
// its neighbours).  Items inside one piece are written out at once; a second kernel joins the
// shared ones by their logsumexps:
//   L = M + ln sum_s exp(L_s - M),  O = sum_s exp(L_s - L) O_s   (M = max_s L_s),
// in the order of the pieces, so the result does not depend on timing.
//
// A CTA is one warp, eight of them to an SM (four at d = 256 over bf16 pages, whose ring is twice as
// large), and waits for no other.  It streams its piece through
// a private ring of three stages filled by TMA, across item and piece boundaries, so that the next
// keys are under way while an item is finished.  SMs do not share HBM evenly (with equal pieces the
// first warp of the 1.07 GB step was done after 130 us and the last after 175), so most of the line
// goes out as one large piece per warp and the rest as small ones, which the warps that are done
// first take over: a warp asks the hardware for the next CTA that has not been launched
// (clusterlaunchcontrol) and does that one's piece.  A page's rows are reached through a tensor map
// over the whole pool; a block of 16 keys never crosses a page (page_size is a multiple of 16).
// Each lane looks up the page of one block, 32 blocks at a time, and issues that block's loads itself.
//
// S = Q K^T, the online softmax and O += P V run on m16n8k16 warp MMAs: 16 rows are too few for a
// tcgen05 tile, and the time goes to reading K and V.  E4M3 codes are converted to f16 (exactly)
// in registers, between the matrix load and the MMA: K's words hold 4 neighbouring elements of d
// of one key, so the MMA's k order is permuted, alike for Q; V's transposed words hold elements
// (2c, 2c + 1) of two keys, which two byte permutes sort into the operands of the even and of the
// odd columns.
//
// Weights enter P V in 16 bits, as one MMA a block takes them: bf16 over bf16 pages, unbiased and off by half
// a step at most, so that O is 0.0021 to 0.0024 from the exact result where its own rounding to bf16 is
// 0.0017; f16 over E4M3 pages (see kPgLift), where nothing of that shows.  More bits would take a second MMA
// for the weights' low part.  The row sums add the weights in fp32 before that rounding.
//
// What it takes (with its merge): 8 sequences of 32768 keys, 8 heads of 128, bf16, 1.07 GB: 181 to 184 us, 5.8 to
// 5.9 TB/s; the copy rate would be 164, the difference is the first loads (5 us), the merge (5 us after the
// last piece) and the stretches' uneven ends.  64 sequences of 0 to 16384 keys: 92 us, 5.1 TB/s.  E4M3 codes,
// 514 MB: 109 to 113 us, 4.6 to 4.7 TB/s.  There the conversions (2.2 cycles of an SMSP) and MMAs (8) of a 4 KB
// block take some 400 cycles one after the other, which would be 11 TB/s; with the tensor pipe 31 % busy and
// IPC 1.6, what bounds it is the chain S, maximum, exponentials, P V of two warps an SMSP.
// 1000 keys: 14 us, all of it latency.  At d = 256 the accumulators and Q do not fit 255 registers: 272 bytes of
// spill stores and 332 of loads a thread (bf16), 224 and 240 (E4M3); the other forms spill none.
#pragma once

#include <climits>
#include <cstdint>

#include "append_kernel.cuh"
#include "decode_kernel.cuh"
#include "paged_ops.cuh"

namespace fa {

constexpr int kPgStages = 3;
constexpr int kPgSurcharge = 2;    // units a new item costs a warp before its first step (Q, output)
constexpr int kPgMinPiece = 4;     // shortest piece of the line, in units
constexpr int kPgMaxWarps = 148 * 8;
// Over E4M3 pages the weights enter P V as f16.  They are formed 2^15 times as large, below f16's largest
// value, so that a weight keeps f16's 11 bits down to 2^-29 of the row's largest (which the row's sum, in fp32,
// counts in full) and is lost below 2^-40 only; formed as they are, keys 17.3 below the largest score would
// be.  The difference to the largest score is formed first, so that no weight passes 2^15, however large
// the scores.
constexpr float kPgLift = 15.f;
constexpr int kPgMergeWarps = 4;   // of one row, at most

// 16-key blocks per step: as many as fill a stage of kPgStageBytes, up to four.  (With 16 KB stages and
// half as many warps the E4M3 step took 130 us instead of 102, the bf16 one 173 instead of 177, and the own
// keys of 64 sequences behind a shared prefix 7 us more.)
constexpr int kPgStageBytes = 8192;
__host__ __device__ constexpr int pg_blocks(int d, bool fp8) {
  const int block = 2 * d * (fp8 ? 1 : 2) * 16;   // a block's K and V
  const int n = kPgStageBytes / block;
  return n < 1 ? 1 : n > 4 ? 4 : n;
}
__host__ __device__ constexpr int pg_step(int d, bool fp8) { return 16 * pg_blocks(d, fp8); }   // keys per step

template <int D, bool kFp8>
struct PgLayout {
  static constexpr int kEsize = kFp8 ? 1 : 2;
  static constexpr int kBlocks = pg_blocks(D, kFp8), kStep = 16 * kBlocks;
  // a block's K tile, then its V tile, as TMA boxes of 16 rows of up to 128 bytes, swizzled by the
  // row width (16-byte piece c of row r at c ^ (r % 8), or c ^ (r / 2 % 4) in 64-byte rows)
  static constexpr int kBoxX = D * kEsize >= 128 ? 128 / kEsize : D;
  static constexpr int kBoxRow = kBoxX * kEsize;    // 128 or 64 bytes
  static constexpr int kBoxes = D / kBoxX;
  static constexpr int kBoxBytes = 16 * kBoxRow;
  static constexpr int kTileBytes = 16 * D * kEsize;
  static constexpr int kBlockBytes = 2 * kTileBytes;
  static constexpr int kStageBytes = kBlocks * kBlockBytes;
  static constexpr int kRingBytes = kPgStages * kStageBytes;
  // then the next piece's handle, the stages' barriers and its own, and the abort flag
  static constexpr int kNextOffset = kRingBytes;
  static constexpr int kBarOffset = kNextOffset + 16;
  static constexpr int kAbortOffset = kBarOffset + (kPgStages + 1) * 8;
  static constexpr int kSmemBytes = 1024 + kAbortOffset + 8;   // rounded up to 1 KB inside the kernel
  static constexpr int kCtasPerSm = 8 * (kSmemBytes + 1024) <= 228 * 1024 ? 8 : 4;
  static_assert(kBoxRow == 128 || kBoxRow == 64, "swizzle row");
  static_assert(32 % kBlocks == 0, "blocks of a step");
  static_assert(kStageBytes % 1024 == 0 && kCtasPerSm * (kSmemBytes + 1024) <= 228 * 1024, "ring");
};
// warps of a full grid: those resident at once
inline int pg_warps(int d, bool fp8) {
  const auto on = [](int per_sm) { return 148 * per_sm; };
  return d == 64    ? on(fp8 ? PgLayout<64, true>::kCtasPerSm : PgLayout<64, false>::kCtasPerSm)
         : d == 128 ? on(fp8 ? PgLayout<128, true>::kCtasPerSm : PgLayout<128, false>::kCtasPerSm)
                    : on(fp8 ? PgLayout<256, true>::kCtasPerSm : PgLayout<256, false>::kCtasPerSm);
}

// The line of work.  Sequence b's items each take kPgSurcharge + steps(b) units.  The host refuses
// a problem whose longest possible line would not fit 31 bits.
struct PgRange {
  int first, steps;   // first step (of kStep keys from key 0) and their number
};
// The keys run from the lowest that the first of the `count` new rows may attend (its band starts
// lowest) to the last key, where the last new row stands.
__host__ __device__ inline PgRange pg_range(int len, int count, int window, int step) {
  PgRange r;
  int lo = 0;
  if (window > 0) {
    const long long l = (long long)len - count - window + 1;
    lo = l > 0 ? int(l) : 0;
  }
  r.first = lo / step;
  r.steps = len > 0 && count > 0 ? (len - 1) / step - r.first + 1 : 0;
  return r;
}
// How the line is cut.  A long line falls into one equal stretch per resident warp, and each stretch
// into a large piece of kPgBigShare of it and one or two small ones; a short line into up to one small
// piece per warp.  Pieces are numbered along the line; the CTAs take the large ones first (taken()), and
// the small ones as they get done.  (The small pieces lie between the large ones, and not all at the
// line's end, so that no item is cut into many more parts than another.)
constexpr float kPgBigShare = 0.7f;
static_assert(kPgBigShare > 0.1f && kPgBigShare < 0.85f && kPgMinPiece >= 2, "a stretch of over 4 kPgMinPiece units "
              "leaves a unit for each of its pieces");
// pieces of a stretch: at d = 256 one small piece, as a partial result is twice as large
__host__ __device__ constexpr int pg_parts(int d) { return d == 256 ? 2 : 3; }
struct PgCut {
  int n, warps, parts, q, rem, q1;   // q1 > 0: stretches of q (the first rem of q + 1) units, large pieces of q1
  __host__ __device__ PgCut(int total, int w, int parts_) {
    warps = w;
    parts = parts_;
    q1 = 0;
    n = (total + kPgMinPiece - 1) / kPgMinPiece;
    if (total > 4 * kPgMinPiece * w) {
      q = total / w;
      rem = total - q * w;
      q1 = int(kPgBigShare * float(q));
      n = parts * w;
    } else {
      n = n < w ? n : w;
      q = total / n;
      rem = total - q * n;
    }
  }
  __host__ __device__ int stretch(int c) const { return q * c + (c < rem ? c : rem); }
  // first unit of a stretch's second small piece (none: past its end)
  __host__ __device__ int second() const { return parts == 3 ? q1 + (q - q1) / 2 : q + 1; }
  // first unit of piece c (0 .. n: n gives the line's end)
  __host__ __device__ int begin(int c) const {
    if (q1 == 0) return stretch(c);
    const int g = c / parts, part = c - parts * g, at = stretch(g);
    return part == 0 ? at : part == 1 ? at + q1 : at + second();
  }
  // the piece that holds unit x
  __host__ __device__ int of(int x) const {
    const int long_ones = rem * (q + 1);
    const int g = x < long_ones ? x / (q + 1) : rem + (x - long_ones) / q;
    if (q1 == 0) return g;
    const int in = x - stretch(g);
    return parts * g + (in < q1 ? 0 : in < second() ? 1 : 2);
  }
  // the piece that CTA c takes
  __host__ __device__ int taken(int c) const {
    if (q1 == 0) return c;
    const int part = c / warps;
    return parts * (c - part * warps) + part;
  }
};

struct PagedParams {
  const __nv_bfloat16* q;   // [B, H, N_q, d]
  __nv_bfloat16* o;         // [B, H, N_q, d]
  float* lse;               // [B, H, N_q] contiguous
  float* o_part;            // [2 pieces][part_rows][d] shared items' partial results (slot 2c: the item
  float* l_part;            // [2 pieces][part_rows]    began before piece c; 2c + 1: it begins in piece c)
  float* o_row;             // [B H N_q][d], [B H N_q]: whole items go here in fp32 instead of o and lse
  float* l_row;             //   (a shared prefix is still to be joined); nullptr otherwise
  const float* o_pre;       // [n_pre][rows of all sequences][d], [n_pre][...]: the prefix's splits
  const float* l_pre;
  const int* table;         // [B, max_pages], rows table_stride apart
  const int* lengths;       // [B]
  const int* counts;        // [B] new rows of each sequence, or nullptr: all N_q
  long long table_stride;
  Strides q_st, o_st;
  long long total_rows;     // B * H * N_q
  int B, H, H_kv, group, Nq;
  int rows, row_blocks;     // rows per K/V head (group * N_q), blocks of 16 of them
  int part_rows;            // min(rows, 16)
  int n_pages, page_size, max_pages;
  int causal, window;
  int warps, n_pre;
  float scale_log2, v_scale;
  unsigned long long wait_limit_ns;
};

// keys of sequence b: its length, no longer than its table row reaches
__device__ __forceinline__ int pg_len(const PagedParams& p, int b) {
  return min(max(p.lengths[b], 0), p.max_pages * p.page_size);
}

// its new rows
__device__ __forceinline__ int pg_count(const PagedParams& p, int b) {
  return p.counts ? min(max(p.counts[b], 0), p.Nq) : p.Nq;
}

// units of one item row (one item) of sequence b
template <int kStep>
__device__ __forceinline__ int pg_units(const PagedParams& p, int b) {
  return kPgSurcharge + pg_range(pg_len(p, b), pg_count(p, b), p.window, kStep).steps;
}
__device__ __forceinline__ int pg_warp_sum(int x) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}
__device__ __forceinline__ int pg_warp_scan(int x, int lane) {   // inclusive
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, m);
    if (lane >= m) x += y;
  }
  return x;
}

// Walks the items of one piece [x0, x1) of the line in order.
template <int kStep>
struct PgCursor {
  int s;            // start of the current item on the line
  int b, j;         // sequence, item of it (K/V head * row_blocks + row block)
  int len, count;
  PgRange r;
  __device__ void load(const PagedParams& p) {
    len = pg_len(p, b);
    count = pg_count(p, b);
    r = pg_range(len, count, p.window, kStep);
  }
  __device__ void next(const PagedParams& p) {
    s += kPgSurcharge + r.steps;
    if (++j == p.H_kv * p.row_blocks) {
      j = 0;
      ++b;
      if (b < p.B) load(p);
    }
  }
  // steps [r0, r1) of the current item that lie in the piece [x0, x1)
  __device__ void part(int x0, int x1, int& r0, int& r1) const {
    r0 = max(x0 - s - kPgSurcharge, 0);
    r1 = max(min(x1 - s - kPgSurcharge, r.steps), r0);
  }
};

// two bytes of a word of E4M3 codes as f16x2: the even or the odd ones
__device__ __forceinline__ uint32_t pg_cvt_even(uint32_t w) { return e4m3_lo_f16x2(byte_perm(w, 0u, 0x0020)); }
__device__ __forceinline__ uint32_t pg_cvt_odd(uint32_t w) { return e4m3_lo_f16x2(byte_perm(w, 0u, 0x0031)); }

// tm_k, tm_v: the page pools as the 4-D tensors (d, page_size, H_kv, n_pages), boxes of
// PgLayout::kBoxX elements x 16 rows.
template <int D, bool kFp8>
__global__ void __launch_bounds__(32, PgLayout<D, kFp8>::kCtasPerSm)
    fa_paged_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const PagedParams p) {
  using Lay = PgLayout<D, kFp8>;
  constexpr int KS = D / 16, NT = D / 8, kBlocks = Lay::kBlocks, kStep = Lay::kStep;
  constexpr float kLn2 = 0.6931471805599453f;
  unsigned char* ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dec_dyn_smem()) + 1023) &
                                                         ~uintptr_t(1023));
  const int lane = threadIdx.x;
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + Lay::kBarOffset);
  volatile int* abort = reinterpret_cast<volatile int*>(ring + Lay::kAbortOffset);
  const uint32_t next_at = smem_u32(ring + Lay::kNextOffset), next_bar = smem_u32(&bars[kPgStages]);
  if (lane == 0) {
    *abort = 0;
    for (int st = 0; st < kPgStages; ++st) mbar_init(smem_u32(&bars[st]), kBlocks);
    mbar_init(next_bar, 1);
    fence_mbar_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  __syncwarp();
  // This grid may be scheduled while the one before it runs.  Nothing that another grid may have written
  // (lengths, tables, q, pages) is read before the wait, and the scratch is not written: what a grid
  // earlier on the stream wrote is visible to a grid that has waited for it, or for one that had, and not
  // already because that one has seen it.  With a shared prefix this grid waits for the prefix's.
  grid_dep_wait();
  // ---- the line of work: every warp adds up the lengths (lane l a run of `per` sequences)
  const int HR = p.H_kv * p.row_blocks;
  const int per = (p.B + 31) >> 5;
  const int sb0 = min(p.B, lane * per), sb1 = min(p.B, sb0 + per);
  int mine = 0;
  for (int b = sb0; b < sb1; ++b) mine += pg_units<kStep>(p, b);
  // the next piece's number, asked for ahead of its use (lane 0)
  auto ask = [&] {
    if (lane == 0) {
      mbar_expect_tx(next_bar, 16);
      cta_steal_async(next_at, next_bar);
    }
  };
  grid_dep_launch_dependents();
  const int run_end = pg_warp_scan(mine, lane), run_at = run_end - mine;
  const int all = __shfl_sync(0xffffffffu, run_end, 31);
  const PgCut cut(all * HR, p.warps, pg_parts(D));
  if (int(blockIdx.x) >= cut.n) return;
  ask();
  int asked = 1;   // requests made
  bool open = true, dry = false;   // the last one is not answered yet; there is no further piece

  // the item that holds a piece's first unit
  auto find = [&](int piece) -> PgCursor<kStep> {
    PgCursor<kStep> c;
    const int x = cut.begin(piece), row_at = x / HR;   // place among one item row's units
    const int run = popc(__ballot_sync(0xffffffffu, sb0 < p.B && run_at <= row_at)) - 1;
    int at = __shfl_sync(0xffffffffu, run_at, run);
    c.b = run * per;
    if (per > 1) {   // which of the run's sequences: 32 at a time
      for (;;) {
        const int b = c.b + lane;
        const int end = at + pg_warp_scan(b < p.B ? pg_units<kStep>(p, b) : 0, lane);
        const int past = popc(__ballot_sync(0xffffffffu, end <= row_at));
        if (past > 0) at = __shfl_sync(0xffffffffu, end, past - 1);
        c.b += past;
        if (past < 32 || c.b >= p.B) break;
      }
      c.b = min(c.b, p.B - 1);   // (no piece begins at the line's end: every piece holds a unit)
    }
    c.load(p);
    const int n = kPgSurcharge + c.r.steps;
    c.j = (x - at * HR) / n;
    c.s = at * HR + c.j * n;
    return c;
  };

  // ---- loads.  The steps of a piece are looked up a batch of 32 blocks at a time, one block a lane.
  // (Everything below has one place in the code, and not one for the start, one for the steady state and
  // one for a change of pieces: a call that finds the instruction cache cold waits for each line of it.
  // With L2 flushed before each call a 1000-key step took 16.4 us so and 18.5 before, the d = 64 draft 26.6
  // and 28.7; the 1.07 GB step in a loop 180 us and 178.)
  int piece_now = -1, piece_load = -1;      // the pieces being worked on and being loaded
  int load_x0 = 0, load_x1 = 0;             // the latter's units
  PgCursor<kStep> begun, ahead;             // its first item, and the one that the look-up has come to
  int ahead_base = 0;                       // its steps before that item
  int batch = 0, turn = 0, left = 0;        // its current batch, that one's next step and number of steps
  int page = -1, place = -1;                // of this lane's block of the batch; place < 0: no such block
  constexpr int kBatch = 32 / kBlocks, kPast = 1 << 30;   // kPast, of a place: past the sequence's length
  // K and V pass through L2 once, unless several row blocks read them: they should not push out the
  // partial results that the merge is to read
  const uint64_t policy = l2_policy(p.row_blocks == 1);
  int issued = 0;
  // The next of my steps into its stage: its blocks' lanes issue, every lane keeps the count.  When the
  // piece is used up the next one is taken over, one ahead of the piece being worked on at most.  False
  // if there is none (for now).
  auto issue = [&]() -> bool {
    while (turn == left) {
      if (left == kBatch) {
        ++batch;
      } else {
        if (dry || piece_load != piece_now) return false;
        int next = int(blockIdx.x);
        if (piece_load >= 0) {
          dry = true;
          if (!__all_sync(0xffffffffu, dec_wait(next_bar, (asked - 1) & 1, abort, p.wait_limit_ns))) return false;
          open = false;
          next = cta_stolen(next_at);
          if (next < 0 || next >= cut.n) return false;
          dry = false;
          fence_proxy_async_smem();   // the answer has been read; its place is next written by the request
          __syncwarp();
          ask();
          ++asked;
          open = true;
        }
        piece_load = cut.taken(next);
        begun = ahead = find(piece_load);
        load_x0 = cut.begin(piece_load), load_x1 = cut.begin(piece_load + 1);
        ahead_base = batch = 0;
      }
      const int blk = 32 * batch + lane, want = blk / kBlocks;
      page = place = -1;
      while (ahead.b < p.B && ahead.s < load_x1) {
        int r0, r1;
        ahead.part(load_x0, load_x1, r0, r1);
        if (want < ahead_base + (r1 - r0)) {
          const int key = (ahead.r.first + r0 + want - ahead_base) * kStep + (blk % kBlocks) * 16;
          const int pg = key / p.page_size;
          place = ((key - pg * p.page_size) >> 4) | ((ahead.j / p.row_blocks) << 11);
          if (key < ahead.len)
            page = p.table[(long long)ahead.b * p.table_stride + pg];
          else
            place |= kPast;
          break;
        }
        ahead_base += r1 - r0;
        ahead.next(p);
      }
      left = popc(__ballot_sync(0xffffffffu, place >= 0)) / kBlocks;
      turn = 0;
    }
    if (lane / kBlocks == turn) {
      // a block past the length reads outside the tensor, as zeros; so does a bad page number
      int from = page;
      if (from < 0 || from >= p.n_pages) {
        if (!(place & kPast)) atomicOr(&g_status, FA_DEVICE_BAD_INDEX);
        from = p.n_pages;
      }
      const int row = (place & 2047) << 4, head = (place & ~kPast) >> 11;
      const uint32_t dst =
          smem_u32(ring + (issued % kPgStages) * Lay::kStageBytes + (lane % kBlocks) * Lay::kBlockBytes);
      const uint32_t bar = smem_u32(&bars[issued % kPgStages]);
      mbar_expect_tx(bar, Lay::kBlockBytes);
#pragma unroll
      for (int c = 0; c < Lay::kBoxes; ++c) {
        tma_load_rows_hint(dst + c * Lay::kBoxBytes, &tm_k, bar, c * Lay::kBoxX, row, head, from, policy);
        tma_load_rows_hint(dst + Lay::kTileBytes + c * Lay::kBoxBytes, &tm_v, bar, c * Lay::kBoxX, row, head, from,
                           policy);
      }
    }
    ++issued;
    ++turn;
    return true;
  };

  const int g = lane >> 2, t = lane & 3;   // MMA fragment row group and column pair
  // Matrix loads: this lane's row and piece of a tile as a byte offset, for K (keys 0-7 and 8-15 of
  // one piece side by side for E4M3, two pieces of keys 0-7 for bf16) and for V (transposed).  As the
  // pieces of a row are swizzled by exclusive or, piece i further along is the offset with i's bits
  // flipped in.
  constexpr int kRowPieces = Lay::kBoxRow / 16;
  auto lane_piece = [&](int kr, int c) -> uint32_t {
    return uint32_t(kr) * Lay::kBoxRow + ((uint32_t(c) ^ (Lay::kBoxRow == 128 ? kr & 7 : (kr >> 1) & 3)) << 4);
  };
  const uint32_t ring_at = smem_u32(ring);
  const uint32_t v_lane = lane_piece(((lane >> 3) & 1) * 8 + (lane & 7), lane >> 4);
  const uint32_t k_lane = kFp8 ? v_lane : lane_piece((lane >> 4) * 8 + (lane & 7), (lane >> 3) & 1);
  auto along = [&](uint32_t at, int i) -> uint32_t {   // i even
    return (at ^ (uint32_t(i % kRowPieces) << 4)) + uint32_t(i / kRowPieces) * Lay::kBoxBytes;
  };
  // byte offset of 16-byte piece c of key row kr of a tile
  auto piece = [&](int kr, int c) -> int {
    if constexpr (Lay::kBoxRow == 128)
      return (c >> 3) * Lay::kBoxBytes + kr * 128 + (((c & 7) ^ (kr & 7)) << 4);
    else
      return kr * 64 + ((c ^ ((kr >> 1) & 3)) << 4);
  };
  // Clears the rows of a block's V tile whose keys lie outside [lo, hi]; whether any other row
  // holds an infinity or NaN (a bf16's full exponent field; the E4M3 codes 0x7f and 0xff).
  auto clean_v = [&](unsigned char* vs, int key0, int lo, int hi) -> bool {
    bool bad = false;
#pragma unroll
    for (int x = 0; x < Lay::kTileBytes / 512; ++x) {
      constexpr int kPieces = D * Lay::kEsize / 16;
      const int c = lane + 32 * x, kr = c / kPieces;
      uint4* at = reinterpret_cast<uint4*>(vs + piece(kr, c % kPieces));
      if (key0 + kr < lo || key0 + kr > hi) {
        *at = make_uint4(0u, 0u, 0u, 0u);
      } else {
        const uint4 w = *at;
        const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (kFp8) {
#pragma unroll
            for (int s = 0; s < 32; s += 8) bad |= ((word[e] >> s) & 0x7fu) == 0x7fu;
          } else {
            bad |= (word[e] & 0x7f80u) == 0x7f80u || (word[e] & 0x7f800000u) == 0x7f800000u;
          }
        }
      }
    }
    fence_proxy_async_smem();   // the stage is next written by TMA
    __syncwarp();               // other lanes read what this one has cleared (a vote orders no memory)
    return __any_sync(0xffffffffu, bad);
  };

  int it = 0;              // my steps done
  bool ok = true, in_item = false;
  PgCursor<kStep> cur;     // the item being worked on, of the piece [x0, x1)
  int x0 = 0, x1 = 0, r0 = 0, r1 = 0, seg_end = 0;   // its steps here, and my count when they are done
  bool begins = false, whole = false;
  int b = 0, hkv = 0, row0 = 0;
  int band_lo[2], band_hi[2], hq[2], qi[2], lo_max = 0, hi_min = 0, any_lo = 0;
  uint32_t qa[KS][4];
  float acc[NT][4], m_run[2], l_run[2];
  for (;;) {
    // fill the ring: steps it .. it + 2 may be in flight, as every lane has left step it - 1
    __syncwarp();
    while (issued < it + kPgStages && issue()) {
    }
    if (!in_item) {
      if (piece_now < 0 || cur.b >= p.B || cur.s >= x1) {
        // the piece is done, and with it all that was issued unless the next one is being loaded
        if (!ok || piece_load == piece_now) break;
        piece_now = piece_load;
        cur = begun;
        x0 = load_x0, x1 = load_x1;
        continue;
      }
      cur.part(x0, x1, r0, r1);
      begins = cur.s >= x0;
      // an item without keys is finished by the warp whose piece it begins in; one whose steps all
      // lie in other pieces is theirs
      if (r1 == r0 && !(cur.r.steps == 0 && begins)) {
        cur.next(p);
        continue;
      }
      whole = r0 == 0 && r1 == cur.r.steps;
      seg_end = it + (r1 - r0);
      in_item = true;
      b = cur.b, hkv = cur.j / p.row_blocks;
      row0 = (cur.j - hkv * p.row_blocks) * kDecRows;
      const int pos0 = cur.len - cur.count;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int r = row0 + g + 8 * hf;
        const __nv_bfloat16* src = nullptr;
        // rows past the end, and padding, stay unmasked and read zero Q; the former are never written, the
        // latter as 0
        band_lo[hf] = INT_MIN;
        band_hi[hf] = INT_MAX;
        hq[hf] = -1;
        if (r < p.rows) {
          const int gh = r / p.Nq;
          qi[hf] = r - gh * p.Nq;
          hq[hf] = hkv * p.group + gh;
          if (qi[hf] < cur.count) {
            dec_band(pos0 + qi[hf], cur.len, p.causal, p.window, band_lo[hf], band_hi[hf]);
            src = p.q + p.q_st.at(b, hq[hf], qi[hf]);
          }
        }
        // Q as the A operand of every k-step: columns 2t, 2t + 1 (+ 8), or for E4M3 the permuted
        // 4t .. 4t + 3
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
          if constexpr (kFp8) {
            uint2 w = {0u, 0u};
            if (src) w = *reinterpret_cast<const uint2*>(src + 16 * kk + 4 * t);
            qa[kk][hf] = bf16x2_to_f16x2_sat_nan(w.x);
            qa[kk][hf + 2] = bf16x2_to_f16x2_sat_nan(w.y);
          } else {
            qa[kk][hf] = src ? ld_global_u32(src + 16 * kk + 2 * t) : 0u;
            qa[kk][hf + 2] = src ? ld_global_u32(src + 16 * kk + 2 * t + 8) : 0u;
          }
        }
        m_run[hf] = -INFINITY;
        l_run[hf] = 0.f;
      }
      // bands move right with the position: the last row's low end and the first row's high end
      // bound the keys that every row may attend, the first row's low end those that any may
      int unused;
      dec_band(cur.len - 1, cur.len, p.causal, p.window, lo_max, unused);
      dec_band(pos0, cur.len, p.causal, p.window, any_lo, hi_min);
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    }
    if (it < seg_end) {
      if (!__all_sync(0xffffffffu, dec_wait(smem_u32(&bars[it % kPgStages]), (it / kPgStages) & 1, abort,
                                            p.wait_limit_ns))) {
        ok = false;
        break;
      }
      const uint32_t st = ring_at + (it % kPgStages) * Lay::kStageBytes;
      const int key0 = (cur.r.first + r1 - (seg_end - it)) * kStep;

      // S = Q K^T: n-tiles of 8 keys
      float s[2 * kBlocks][4];
#pragma unroll
      for (int n = 0; n < 2 * kBlocks; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < KS; kk += kFp8 ? 2 : 1) {
#pragma unroll
        for (int bl = 0; bl < kBlocks; ++bl) {
          const uint32_t ks = st + bl * Lay::kBlockBytes + k_lane;
          uint32_t kf[4];
          if constexpr (kFp8) {
            // matrices: keys 0-7 | 8-15 of columns 16kk .., then of columns 16(kk + 1) ..: two k-steps
            ldmatrix_x4_at(kf, along(ks, kk));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              mma_16816_free<true>(s[2 * bl], qa[kk + h], e4m3_lo_f16x2(kf[2 * h]), e4m3_hi_f16x2(kf[2 * h]));
              mma_16816_free<true>(s[2 * bl + 1], qa[kk + h], e4m3_lo_f16x2(kf[2 * h + 1]),
                                   e4m3_hi_f16x2(kf[2 * h + 1]));
            }
          } else {
            // matrices: keys 0-7 | 8-15  x  columns 16kk + 0-7 | 8-15
            ldmatrix_x4_at(kf, along(ks, 2 * kk));
            mma_16816_free<false>(s[2 * bl], qa[kk], kf[0], kf[1]);
            mma_16816_free<false>(s[2 * bl + 1], qa[kk], kf[2], kf[3]);
          }
        }
      }
      // mask keys outside a row's band (and past the length)
      const bool need_mask = key0 < lo_max || key0 + kStep - 1 > hi_min;
      if (need_mask) {
#pragma unroll
        for (int n = 0; n < 2 * kBlocks; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int key = key0 + 8 * n + 2 * t + (c & 1);
            if (key < band_lo[c >> 1] || key > band_hi[c >> 1]) s[n][c] = -INFINITY;
          }
      }
      // online softmax per row, with the running max m in unscaled scores and weights
      // 2^((s - m) scale log2 e): the four lanes of a row group share it
      float alpha[2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float mx = fmaxf(s[0][2 * hf], s[0][2 * hf + 1]);
#pragma unroll
        for (int n = 1; n < 2 * kBlocks; ++n) mx = fmaxf(mx, fmaxf(s[n][2 * hf], s[n][2 * hf + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float m_new = fmaxf(m_run[hf], mx);
        const float m_fin = m_new == -INFINITY ? 0.f : m_new;   // a row with no key yet stays at 0
        const float m_use = -m_fin * p.scale_log2;
        alpha[hf] = ex2_approx((m_run[hf] - m_fin) * p.scale_log2);   // exactly 1 while the max stands
        m_run[hf] = m_new;
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < 2 * kBlocks; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = s[n][2 * hf + e];
            s[n][2 * hf + e] =
                ex2_approx(kFp8 ? (x - m_fin) * p.scale_log2 + kPgLift : x * p.scale_log2 + m_use);
            sum += s[n][2 * hf + e];
          }
        l_run[hf] = l_run[hf] * alpha[hf] + sum;   // this lane's share; summed over the group at the end
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {   // some row's max has grown
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          acc[j][0] *= alpha[0];
          acc[j][1] *= alpha[0];
          acc[j][2] *= alpha[1];
          acc[j][3] *= alpha[1];
        }
      }
      // O += P V; P (bf16, or f16) is the A operand straight from the S fragments
#pragma unroll
      for (int bl = 0; bl < kBlocks; ++bl) {
        const uint32_t vb = st + bl * Lay::kBlockBytes + Lay::kTileBytes + v_lane;
        unsigned char* vs = ring + (it % kPgStages) * Lay::kStageBytes + bl * Lay::kBlockBytes + Lay::kTileBytes;
        const int bkey = key0 + 16 * bl;
        // 0 x NaN is NaN: V rows that no row may attend are cleared before the product, and if a
        // key that only some rows may attend holds infinities or NaN, the block's product is formed
        // key by key, so that they reach the rows that attend it alone
        if (need_mask && clean_v(vs, bkey, any_lo, cur.len - 1)) {
          for (int kk = 0; kk < 16; ++kk) {
            const int key = bkey + kk, src = (lane & ~3) | ((kk & 7) >> 1);
            const float* lo = s[2 * bl];
            const float* hi = s[2 * bl + 1];
            const float w0 = kk < 8 ? (kk & 1 ? lo[1] : lo[0]) : (kk & 1 ? hi[1] : hi[0]);
            const float w1 = kk < 8 ? (kk & 1 ? lo[3] : lo[2]) : (kk & 1 ? hi[3] : hi[2]);
            const float p0 = __shfl_sync(0xffffffffu, w0, src), p1 = __shfl_sync(0xffffffffu, w1, src);
            const bool on0 = key >= band_lo[0] && key <= band_hi[0], on1 = key >= band_lo[1] && key <= band_hi[1];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              float v0, v1;   // the key's elements of this lane's two columns of tile j
              if constexpr (kFp8) {
                // tiles 2c, 2c + 1: columns 16c + 4t, + 2 and 16c + 4t + 1, + 3
                const uint32_t w = *reinterpret_cast<const uint32_t*>(vs + piece(kk, j >> 1) + 4 * t);
                f16x2_to_f32(j & 1 ? pg_cvt_odd(w) : pg_cvt_even(w), v0, v1);
              } else {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(vs + piece(kk, j) + 4 * t);
                v0 = app_lo(w);
                v1 = app_hi(w);
              }
              acc[j][0] += on0 ? p0 * v0 : 0.f;
              acc[j][1] += on0 ? p0 * v1 : 0.f;
              acc[j][2] += on1 ? p1 * v0 : 0.f;
              acc[j][3] += on1 ? p1 * v1 : 0.f;
            }
          }
          continue;
        }
        const uint32_t pa[4] = {dec_pack<kFp8>(s[2 * bl][0], s[2 * bl][1]), dec_pack<kFp8>(s[2 * bl][2], s[2 * bl][3]),
                                dec_pack<kFp8>(s[2 * bl + 1][0], s[2 * bl + 1][1]),
                                dec_pack<kFp8>(s[2 * bl + 1][2], s[2 * bl + 1][3])};
        if constexpr (kFp8) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            // transposed matrices: keys 0-7 | 8-15 of code pairs 32c .., then of 32c + 16 ..
            uint32_t vf[4];
            ldmatrix_x4_trans_at(vf, along(vb, 2 * c));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              mma_16816_free<true>(acc[4 * c + 2 * h], pa, pg_cvt_even(vf[2 * h]), pg_cvt_even(vf[2 * h + 1]));
              mma_16816_free<true>(acc[4 * c + 2 * h + 1], pa, pg_cvt_odd(vf[2 * h]), pg_cvt_odd(vf[2 * h + 1]));
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            uint32_t vf[4];   // transposed matrices: keys 0-7 | 8-15  x  columns 16j + 0-7 | 8-15
            ldmatrix_x4_trans_at(vf, along(vb, 2 * j));
            mma_16816_free<false>(acc[2 * j], pa, vf[0], vf[1]);
            mma_16816_free<false>(acc[2 * j + 1], pa, vf[2], vf[3]);
          }
        }
      }
      ++it;
      if (it < seg_end) continue;
    }

    // ---- the item's rows, or this piece's part of them
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      float l = l_run[hf];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (hq[hf] < 0) continue;
      if (qi[hf] >= cur.count) {   // padding
        l = 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[j][2 * hf] = acc[j][2 * hf + 1] = 0.f;
      }
      // a row without keys, or whose every key scored -inf, has l = 0; one with a NaN score is NaN
      float inv = l == 0.f ? 0.f : 1.f / l;
      if constexpr (kFp8) inv *= p.v_scale;
      const float lse =
          l == 0.f ? -INFINITY : (m_run[hf] * p.scale_log2 + (lg2_approx(l) - (kFp8 ? kPgLift : 0.f))) * kLn2;
      const long long grow = ((long long)b * p.H + hq[hf]) * p.Nq + qi[hf];
      if (whole && !p.o_row) {
        __nv_bfloat16* dst = p.o + p.o_st.at(b, hq[hf], qi[hf]);
        if constexpr (kFp8) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint2 w;
            w.x = pack_bf16x2(acc[2 * c][2 * hf] * inv, acc[2 * c + 1][2 * hf] * inv);
            w.y = pack_bf16x2(acc[2 * c][2 * hf + 1] * inv, acc[2 * c + 1][2 * hf + 1] * inv);
            *reinterpret_cast<uint2*>(dst + 16 * c + 4 * t) = w;
          }
        } else {
#pragma unroll
          for (int j = 0; j < NT; ++j)
            *reinterpret_cast<uint32_t*>(dst + 8 * j + 2 * t) =
                pack_bf16x2(acc[j][2 * hf] * inv, acc[j][2 * hf + 1] * inv);
        }
        if (t == 0) p.lse[grow] = lse;
      } else {
        const long long prow = whole ? grow : (2ll * piece_now + (begins ? 1 : 0)) * p.part_rows + g + 8 * hf;
        float* dst = (whole ? p.o_row : p.o_part) + prow * D;
        if constexpr (kFp8) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
            *reinterpret_cast<float4*>(dst + 16 * c + 4 * t) =
                make_float4(acc[2 * c][2 * hf] * inv, acc[2 * c + 1][2 * hf] * inv, acc[2 * c][2 * hf + 1] * inv,
                            acc[2 * c + 1][2 * hf + 1] * inv);
        } else {
#pragma unroll
          for (int j = 0; j < NT; ++j)
            *reinterpret_cast<float2*>(dst + 8 * j + 2 * t) =
                make_float2(acc[j][2 * hf] * inv, acc[j][2 * hf + 1] * inv);
        }
        if (t == 0) (whole ? p.l_row : p.l_part)[prow] = lse;
      }
    }
    cur.next(p);
    in_item = false;
  }
  // after an abort, what is still in flight lands before the shared memory is released
  if (lane == 0 && open) mbar_wait_drain(next_bar, (asked - 1) & 1, p.wait_limit_ns);
  if (lane == 0)
    for (int j = it; j < issued; ++j)
      mbar_wait_drain(smem_u32(&bars[j % kPgStages]), (j / kPgStages) & 1, p.wait_limit_ns);
}

__device__ __forceinline__ float* merge_smem() { return reinterpret_cast<float*>(dec_dyn_smem()); }
constexpr int pg_merge_smem(int d) { return kPgMergeWarps * (d + 2) * 4; }

// Join the partial results of every output row, one CTA per row: the pieces that share its item
// (or its whole item's fp32 row), and the prefix's splits.  A row whose whole item was written by
// one warp, with no prefix, is left alone.  Source n of a row: n < n_own its own keys' partials,
// then the prefix's splits.  The warps take groups of eight sources in turn, load their L and rows
// together and join them by a running maximum; the warps are then joined in shared memory.
template <int D, int kStep>
__global__ void __launch_bounds__(32 * kPgMergeWarps) fa_paged_merge_kernel(const PagedParams p) {
  constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;
  constexpr int C = D / 32, kAtOnce = 8;
  float* sm = merge_smem();   // [warps][D], then m and l of each warp
  const int grow = int(blockIdx.x), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warps = int(blockDim.x) >> 5;
  const int bh = grow / p.Nq, i = grow - bh * p.Nq;
  const int b = bh / p.H, hq = bh - b * p.H;
  const int hkv = hq / p.group, r = (hq - hkv * p.group) * p.Nq + i;
  const int HR = p.H_kv * p.row_blocks;
  // not even the lengths are read before the wait, though the grid before this one has seen them (see there)
  grid_dep_wait();
  // the row's item on the line, from the lengths alone
  int before = 0, all = 0;
  for (int x = lane; x < p.B; x += 32) {
    const int u = pg_units<kStep>(p, x);
    all += u;
    before += x < b ? u : 0;
    // (reported here, as any CTA of the grid before may be taken over, and then never runs)
    if (grow == 0 && (p.lengths[x] > p.max_pages * p.page_size || (p.counts && p.counts[x] != pg_count(p, x))))
      atomicOr(&g_status, FA_DEVICE_BAD_INDEX);
  }
  before = pg_warp_sum(before);
  const int total = pg_warp_sum(all) * HR, n = pg_units<kStep>(p, b);
  const int s = before * HR + n * (hkv * p.row_blocks + r / kDecRows);
  const PgCut cut(total, p.warps, pg_parts(D));
  const int steps = n - kPgSurcharge;
  // an item's steps begin after its surcharge: pieces that hold only surcharge wrote nothing
  const int c_item = cut.of(s);
  const int c0 = steps > 0 ? cut.of(s + kPgSurcharge) : c_item;
  const int c1 = steps > 0 ? cut.of(s + n - 1) : c_item;
  const bool whole = c0 == c1;
  const int n_own = whole ? 1 : c1 - c0 + 1;
  const int n_src = i < pg_count(p, b) ? n_own + p.n_pre : 0;   // padding joins nothing: O = 0, L = -inf
  if (whole && !p.o_row) return;
  // the prefix's rows of one K/V head: those of all sequences, in order
  const long long pre_row = ((long long)hkv * p.B + b) * p.rows + r;
  float mx = -INFINITY, sum = 0.f;
  float acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = 0.f;
  for (int s0 = warp * kAtOnce; s0 < n_src; s0 += warps * kAtOnce) {
    float L[kAtOnce], x[kAtOnce][C];
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) {
      const int src = s0 + e;
      L[e] = -INFINITY;
      if (src < n_src) {
        const float *o, *l;
        long long at;
        if (src >= n_own) {
          at = (long long)(src - n_own) * p.total_rows + pre_row;
          o = p.o_pre, l = p.l_pre;
        } else if (whole) {
          at = grow;
          o = p.o_row, l = p.l_row;
        } else {
          const int c = c0 + src;
          at = (2ll * c + (c == c_item ? 1 : 0)) * p.part_rows + r % kDecRows;
          o = p.o_part, l = p.l_part;
        }
        L[e] = l[at];
        o += at * D + lane * C;
        if constexpr (C % 4 == 0) {
#pragma unroll
          for (int c = 0; c < C; c += 4) {
            const float4 w = *reinterpret_cast<const float4*>(o + c);
            x[e][c] = w.x, x[e][c + 1] = w.y, x[e][c + 2] = w.z, x[e][c + 3] = w.w;
          }
        } else {
          const float2 w = *reinterpret_cast<const float2*>(o);
          x[e][0] = w.x, x[e][1] = w.y;
        }
      }
    }
    float m_new = mx;
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) m_new = fmaxf(m_new, L[e]);
    const float m_use = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = ex2_approx((mx - m_use) * kLog2e);   // 0 for the first
    mx = m_new;
    sum *= alpha;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] *= alpha;
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e)
      if (s0 + e < n_src) {
        const float w = ex2_approx((L[e] - m_use) * kLog2e);
        sum += w;
        if (L[e] != -INFINITY) {   // a source without keys has weight 0 and may hold no row
#pragma unroll
          for (int c = 0; c < C; ++c) acc[c] += w * x[e][c];
        }
      }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) sm[warp * D + lane * C + c] = acc[c];
  if (lane == 0) {
    sm[kPgMergeWarps * D + warp] = mx;
    sm[kPgMergeWarps * D + kPgMergeWarps + warp] = sum;
  }
  __syncthreads();
  const float* ml = sm + kPgMergeWarps * D;
  mx = ml[0];
  for (int w = 1; w < warps; ++w) mx = fmaxf(mx, ml[w]);
  const float m_use = mx == -INFINITY ? 0.f : mx;
  float scale[kPgMergeWarps];
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kPgMergeWarps; ++w) {
    scale[w] = w < warps ? ex2_approx((ml[w] - m_use) * kLog2e) : 0.f;
    if (w < warps) sum += scale[w] * ml[kPgMergeWarps + w];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  __nv_bfloat16* dst = p.o + p.o_st.at(b, hq, i);
  for (int e = 2 * int(threadIdx.x); e < D; e += 2 * int(blockDim.x)) {
    float o0 = 0.f, o1 = 0.f;
#pragma unroll
    for (int w = 0; w < kPgMergeWarps; ++w)
      if (w < warps) {
        o0 += scale[w] * sm[w * D + e];
        o1 += scale[w] * sm[w * D + e + 1];
      }
    *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(o0 * inv, o1 * inv);
  }
  if (threadIdx.x == 0) p.lse[grow] = sum == 0.f ? -INFINITY : mx + lg2_approx(sum) * kLn2;
}

}  // namespace fa
