// Attention of a whole batch's query rows over one prefix that all its sequences share.
//
// The prefix's keys lie in pages of the cache, the same ones for every sequence, and every row
// attends all of them: for one K/V head this is a dense product of all R = B * group * N_q rows with
// the prefix, read once for the whole batch.  The rows' own keys are the paged kernel's; the two
// results are joined by their logsumexps (fa_paged_merge_kernel).  With many rows the two products
// bound the kernel, so they run on tcgen05 MMAs; with up to 128 rows, reading K and V does.
//
// One CTA takes 256 rows (or, with R <= 128, all of them) and one split of the prefix's key tiles,
// and writes its rows' normalised O and L as fp32 partial results.  Its two softmax warpgroups
// ("streams") keep the tensor pipe busy in turn (one's products run while the other's exponentials
// do):
//   rows form   stream w owns rows 128 w .. of the CTA, every key tile serves both;
//   keys form   (R <= 128) both streams share the rows; stream w takes every second key tile, and
//               writes a partial result of its own.
// At d = 256 one stream of 128 rows fits tensor memory, with tiles of 64 keys; its S has two buffers, so
// that the tensor pipe forms the next tile's S while the softmax works on this one's.
//   warp 8       TMA: K_0, then K_{t+1}, V_t for t = 0, 1, ..., through a four-slot ring.  A tile is
//                made of boxes of up to 128 rows that never cross a page; each lane looks up the
//                page of one box, a tile ahead.
//   warp 9       MMA issue: S = Q K^T into TMEM, O += P V with P from TMEM.
//   warps 0-7    softmax: thread t of a stream owns row t (TMEM lane t): running max and sum, P packed
//                to 16 bits over the S columns, O rescaled only when a row's max grows by more than
//                2^8 (E4M3 pages: 2^4), and at the end O / l and L.
//   warps 10-13  (E4M3 pages; at d = 256 warps 4-7 too: 73.5 us instead of 77.6 for 16 heads of 68 rows over
//                10140 keys) convert each tile's codes, which TMA leaves in a ring of their own, to f16
//                operand tiles; Q is rounded to f16 after clamping to its range, P is f16.
// Rows: row r of a head is sequence r / (group N_q), query head r / N_q % group, new row r % N_q.  A
// 128-row tile holds as many whole sequences as fit, so that one TMA box {64, N_q, group, sequences}
// per 64 columns loads it; sequences of more than 128 rows are cut anywhere, and the softmax warps
// gather their Q rows.  (Gathering all Q took 6 to 9 us of a call.)
// What it takes: 64 sequences of 8 rows a head over 32768 keys of 8 heads (135 MB, 69 GFLOP) 71 us of a
// call's 101 to 104, the tensor pipe busy 53 % of them.  There the chain S, exponentials, P V of each stream, which
// the other stream covers in part, bounds it; with few rows the conversion (E4M3) or reading K and V.  S
// in two buffers at d = 256 brought 60 sequences of 8 rows over 20000 keys from 97 to 79 us.
// All exponentials run on MUFU, which keeps a partial result's L good to fp32 and NaN scores NaN.  (With a
// degree-4 polynomial on the FMA pipe for 4, 6 or 8 of every 16 pairs the call took 94.3, 94.3 and 95.4 us
// instead of 95.8, an E4M3 batch of 32 sequences over 8192 keys 48.9, 47.8 and 49.4 instead of 48.1, each over
// the same inputs again and again.)
// The bf16 forms use 165 registers (d = 256: 104) and spill none; with E4M3 pages 14 warps leave 128 registers a
// thread, and the d = 64 and 128 forms spill 24 bytes of stores and 48 of loads.
// Keys past the prefix's end in its last tile get weight 0; their V rows are cleared first, as the
// page may hold anything there (0 x NaN is NaN).
#pragma once

#include "fwd_kernel.cuh"
#include "paged_kernel.cuh"

namespace fa {

constexpr int kPfSlots = 4;
constexpr int kPfRaw = 2;
constexpr int kPfWarpTma = 8, kPfWarpMma = 9;
// O is rescaled when a row's maximum has grown by more than 2^this since it was last.  Over E4M3 pages, whose
// weights enter P V as f16, they are formed 2^kPfLift times as large (see kPgLift): those of a maximum that
// has grown unseen stay below f16's largest value, and weights keep f16's 11 bits down to 2^-25 of the row's
// largest and are lost below 2^-36 only.
__host__ __device__ constexpr float pf_growth(bool fp8) { return fp8 ? 4.f : kRescaleThreshold; }
constexpr float kPfLift = 11.f;
static_assert(pf_growth(true) + kPfLift <= 15.f, "weights within f16");
__host__ __device__ constexpr int pf_streams(int d) { return d == 256 ? 1 : 2; }
__host__ __device__ constexpr int pf_keys(int d) { return d == 256 ? 64 : 128; }   // keys per tile
__host__ __device__ constexpr int pf_threads(bool fp8) { return fp8 ? 448 : 320; }

struct PrefixParams {
  const __nv_bfloat16* q;   // [B, H, N_q, d]
  float* o_pre;             // [partials][H_kv][R][d]
  float* l_pre;             // [partials][H_kv][R]
  const int* pages;         // page numbers of the prefix
  Strides q_st;
  int R, rows, Nq, group, H_kv;      // rows per K/V head: R of all sequences, `rows` of one
  int tile_rows, tile_seqs;          // rows of a tile, and its sequences (0: tiles of 128 gathered rows)
  int len, n_pages, page_size, box_rows;
  int n_tiles, tiles_per_split, n_splits, row_groups;
  int by_keys;              // keys form
  float scale_log2, v_scale;
  unsigned long long wait_limit_ns;
};

template <int D, bool kFp8>
struct PrefixSmem {
  static constexpr int kStreams = pf_streams(D), kKeys = pf_keys(D);
  static constexpr int kConvert = kStreams == 1 ? 256 : 128;   // threads that convert codes
  static constexpr uint32_t kQBytes = 128 * D * 2, kTileBytes = kKeys * D * 2;
  static constexpr uint32_t kRawBytes = kFp8 ? kKeys * D : 0;
  static constexpr uint32_t kQ = 0, kSlot = kStreams * kQBytes, kRawAt = kSlot + kPfSlots * kTileBytes;
  // 4 KB a softmax warp for turning its output rows: the raw ring, which is free by then, or room of its own
  static constexpr uint32_t kTurn = kRawAt, kTurnBytes = 4 * kStreams * 4096;
  static constexpr uint32_t kBars = kRawAt + (kFp8 ? kPfRaw * kRawBytes : kTurnBytes);
  static_assert(!kFp8 || D == 64 || kPfRaw * kRawBytes >= kTurnBytes, "room to turn output rows");
  // barriers: q_full, slot full / empty, raw full / empty, s_full, p_full, o_final per stream (with one
  // stream, s_full and p_full per S buffer, and o_final[1] after every tile's P V), drain, and q_ready
  // (E4M3: Q is f16)
  static constexpr int kQFull = 0, kFull = 1, kEmpty = kFull + kPfSlots, kRawFull = kEmpty + kPfSlots,
                       kRawEmpty = kRawFull + kPfRaw, kSFull = kRawEmpty + kPfRaw, kPFull = kSFull + 2,
                       kOFinal = kPFull + 2, kDrain = kOFinal + 2, kQReady = kDrain + 1,
                       kNumBars = kQReady + 1;
  static constexpr uint32_t kTmemBase = kBars + 8 * kNumBars, kAbort = kTmemBase + 4;
  static constexpr uint32_t kBytes = kAbort + 4;
  static constexpr uint32_t kAlloc = kBytes + 1024 > 120 * 1024 ? kBytes + 1024 : 120 * 1024;   // one CTA an SM
  static_assert(kAlloc <= 232448, "prefix shared memory exceeds 227 KB");
};

// load order of the ring: K_0, then K_{t+1}, V_t (V_t alone for the last tile)
__host__ __device__ constexpr int pf_k_load(int t) { return t == 0 ? 0 : 2 * t - 1; }
__host__ __device__ constexpr int pf_v_load(int t, int n) { return t + 1 < n ? 2 * t + 2 : 2 * t + 1; }

template <int D, bool kFp8>
__global__ void __launch_bounds__(pf_threads(kFp8), 1)
    fa_prefix_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const PrefixParams p) {
  using Sm = PrefixSmem<D, kFp8>;
  constexpr int kKeys = Sm::kKeys, kChunks = D / 64, kStreams = Sm::kStreams;
  constexpr uint32_t kChunkQ = 128 * 128, kChunkKv = kKeys * 128;   // bytes of a 64-column chunk
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dec_dyn_smem()) + 1023) &
                                                         ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return base + Sm::kBars + 8 * i; };
  volatile int* abort = reinterpret_cast<volatile int*>(smem + Sm::kAbort);
  const uint64_t lim = p.wait_limit_ns;

  // this CTA's split, rows and head: CTAs of one split and head are neighbours (their keys meet in L2)
  int bid = blockIdx.x;
  const int rg = bid % p.row_groups;
  bid /= p.row_groups;
  const int split = bid % p.n_splits, hkv = bid / p.n_splits;
  const int tile0 = rg * (p.by_keys ? 1 : kStreams), row0 = tile0 * p.tile_rows;
  const int t_begin = split * p.tiles_per_split;
  const int n = min(p.n_tiles - t_begin, p.tiles_per_split);   // >= 1
  // streams with work, and their tiles (in the keys form tile t is stream t % 2's)
  const bool two = kStreams == 2 && (p.by_keys ? n > 1 : row0 + p.tile_rows < p.R);
  const int q_tiles = two && !p.by_keys ? 2 : 1;
  auto tiles_of = [&](int w) { return p.by_keys && kStreams == 2 ? (n + 1 - w) / 2 : (w == 0 || two ? n : 0); };

  if (threadIdx.x == 0) {
    *abort = 0;
    mbar_init(bar(Sm::kQFull), p.tile_seqs ? 1 : 128 * kStreams);
    mbar_init(bar(Sm::kQReady), 128 * kStreams);
    for (int s = 0; s < kPfSlots; ++s) {
      mbar_init(bar(Sm::kFull + s), kFp8 ? Sm::kConvert : 1);
      mbar_init(bar(Sm::kEmpty + s), 1);
    }
    for (int s = 0; s < kPfRaw; ++s) {
      mbar_init(bar(Sm::kRawFull + s), 1);
      mbar_init(bar(Sm::kRawEmpty + s), Sm::kConvert);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(bar(Sm::kSFull + w), 1);
      mbar_init(bar(Sm::kPFull + w), 128);
      mbar_init(bar(Sm::kOFinal + w), 1);
    }
    mbar_init(bar(Sm::kDrain), 1);
    fence_mbar_init();
  }
  if (warp == kPfWarpTma) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    __syncwarp();
    tmem_alloc(base + Sm::kTmemBase, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<const volatile uint32_t*>(smem + Sm::kTmemBase);
  // the grid before this one has ended (q's producer, the append); the next one, the own keys', may be
  // scheduled and waits for this one in its turn
  grid_dep_wait();
  grid_dep_launch_dependents();

  if (warp == kPfWarpTma) {
    // ------------------------------------------------------------------ TMA producer
    constexpr int kRing = kFp8 ? kPfRaw : kPfSlots;
    constexpr int full0 = kFp8 ? Sm::kRawFull : Sm::kFull, empty0 = kFp8 ? Sm::kRawEmpty : Sm::kEmpty;
    constexpr uint32_t at0 = kFp8 ? Sm::kRawAt : Sm::kSlot;
    constexpr uint32_t bytes = kFp8 ? Sm::kRawBytes : Sm::kTileBytes;
    constexpr int kBoxX = kFp8 ? (D >= 128 ? 128 : 64) : 64;
    constexpr uint32_t kRowBytes = kBoxX * (kFp8 ? 1 : 2);
    const int boxes = kKeys / p.box_rows;   // at most 8
    // place of box `lane` of tile t: its page (outside the pool past the prefix's end, or when the
    // number is bad: reads as zeros) and row
    auto place = [&](int t, int& page, int& row) {
      page = p.n_pages;
      row = 0;
      const int key = (t_begin + t) * kKeys + lane * p.box_rows;
      if (t < n && lane < boxes && key < p.len) {
        const int at = key / p.page_size;
        row = key - at * p.page_size;
        page = p.pages[at];
      }
    };
    auto load = [&](int L, const CUtensorMap* map, int page, int row, bool inside) -> bool {
      const int slot = L % kRing;
      if (!__all_sync(0xffffffffu, mbar_wait(bar(empty0 + slot), ((L / kRing) & 1) ^ 1, abort, lim))) return false;
      if (lane == 0) mbar_expect_tx(bar(full0 + slot), bytes);
      __syncwarp();
      if (lane < boxes) {
        if (page < 0 || page >= p.n_pages) {
          if (inside) atomicOr(&g_status, FA_DEVICE_BAD_INDEX);
          page = p.n_pages;
        }
        const uint32_t dst = base + at0 + slot * bytes + lane * p.box_rows * kRowBytes;
#pragma unroll
        for (int c = 0; c < D / kBoxX; ++c)
          tma_load_rows(dst + c * kKeys * kRowBytes, map, bar(full0 + slot), c * kBoxX, row, hkv, page);
      }
      return true;
    };
    if (p.tile_seqs && lane == 0) {
      const uint32_t bytes_q = uint32_t(p.tile_rows) * D * 2;   // a box past the last sequence is filled with zeros
      mbar_expect_tx(bar(Sm::kQFull), q_tiles * bytes_q);
      for (int w = 0; w < q_tiles; ++w)
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          tma_load_rows(base + Sm::kQ + w * Sm::kQBytes + c * kChunkQ, &tm_q, bar(Sm::kQFull), c * 64, 0,
                        hkv * p.group, (tile0 + w) * p.tile_seqs);
    }
    int issued = 0, page0, row0_, page1, row1;
    auto in = [&](int t) { return t < n && (t_begin + t) * kKeys + lane * p.box_rows < p.len; };
    place(0, page0, row0_);
    place(1, page1, row1);
    bool ok = load(0, &tm_k, page0, row0_, in(0));
    if (ok) issued = 1;
    for (int t = 0; ok && t < n; ++t) {
      int page2, row2;
      place(t + 2, page2, row2);
      if (t + 1 < n) {
        ok = load(pf_k_load(t + 1), &tm_k, page1, row1, in(t + 1));
        if (!ok) break;
        ++issued;
      }
      ok = load(pf_v_load(t, n), &tm_v, page0, row0_, in(t));
      if (!ok) break;
      ++issued;
      page0 = page1, row0_ = row1;
      page1 = page2, row1 = row2;
    }
    // every copy lands before the CTA may exit
    if (p.tile_seqs && lane == 0) mbar_wait_drain(bar(Sm::kQFull), 0, lim);
    if (lane == 0)
      for (int L = max(0, issued - kRing); L < issued; ++L)
        mbar_wait_drain(bar(full0 + L % kRing), (L / kRing) & 1, lim);
    __syncwarp();
  } else if (warp == kPfWarpMma) {
    // ------------------------------------------------------------------ MMA issuer
    auto wait = [&](int i, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar(i), parity, abort, lim));
    };
    constexpr uint32_t kF16 = ~((1u << 7) | (1u << 10));   // A and B f16 instead of bf16
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, kKeys, false, false) & (kFp8 ? kF16 : ~0u);
    constexpr uint32_t idesc_o = idesc_bf16_f32(128, D, false, true) & (kFp8 ? kF16 : ~0u);
    const uint64_t dq0 = sw128_desc(base + Sm::kQ, 16, 1024);
    const uint64_t dk0 = sw128_desc(base + Sm::kSlot, 16, 1024);
    const uint64_t dv0 = sw128_desc(base + Sm::kSlot, kChunkKv, 1024);
    auto full = [&](int L) { return wait(Sm::kFull + L % kPfSlots, (L / kPfSlots) & 1); };
    auto release = [&](int L) { mma_commit_w(bar(Sm::kEmpty + L % kPfSlots)); };
    auto issue_s = [&](int w, int L) {
      const uint64_t dk = desc_advance(dk0, (L % kPfSlots) * Sm::kTileBytes);
      const uint64_t dq = desc_advance(dq0, (p.by_keys || kStreams == 1 ? 0 : w) * Sm::kQBytes);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_bf16_ss_w(tmem + w * 128, desc_advance(dq, (kk >> 2) * kChunkQ + (kk & 3) * 32),
                      desc_advance(dk, (kk >> 2) * kChunkKv + (kk & 3) * 32), idesc_s, kk > 0);
      mma_commit_w(bar(Sm::kSFull + w));
    };
    int pv[2] = {0, 0};
    auto issue_pv = [&](int w, int L) {
      const uint64_t dv = desc_advance(dv0, (L % kPfSlots) * Sm::kTileBytes);
#pragma unroll
      for (int kk = 0; kk < kKeys / 16; ++kk)
        mma_bf16_ts_w(tmem + 256 + w * 128, tmem + w * 128 + kk * 8, desc_advance(dv, kk * 2048), idesc_o,
                      kk > 0 ? 1u : uint32_t(pv[w] > 0));
      if (++pv[w] == tiles_of(w)) mma_commit_w(bar(Sm::kOFinal + w));
    };
    // one stream: buffer t % 2 holds tile t's S, then its P
    auto issue_pv_one = [&](int t, int L) {
      const uint64_t dv = desc_advance(dv0, (L % kPfSlots) * Sm::kTileBytes);
#pragma unroll
      for (int kk = 0; kk < kKeys / 16; ++kk)
        mma_bf16_ts_w(tmem + 256, tmem + (t & 1) * 128 + kk * 8, desc_advance(dv, kk * 2048), idesc_o,
                      kk > 0 ? 1u : uint32_t(t > 0));
      mma_commit_w(bar(Sm::kOFinal + 1));
      if (t + 1 == n) mma_commit_w(bar(Sm::kOFinal));
    };
    // V_t has landed; rows past the prefix's end are cleared (E4M3: the conversion did)
    auto v_ready = [&](int t) -> bool {
      const int L = pf_v_load(t, n);
      if (!full(L)) return false;
      const int valid = p.len - (t_begin + t) * kKeys;
      if (!kFp8 && valid < kKeys) {
        for (int c = 0; c < kChunks; ++c)
          for (int x = valid * 8 + lane; x < kKeys * 8; x += 32)   // whole rows: the swizzle moves nothing out of them
            st_shared_v4(base + Sm::kSlot + (L % kPfSlots) * Sm::kTileBytes + c * kChunkKv + x * 16, 0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
      }
      return true;
    };
    bool ok = wait(kFp8 ? Sm::kQReady : Sm::kQFull, 0) && full(0);
    if (ok) {
      tc_fence_after();
      issue_s(0, 0);
      if (kStreams == 2 && two && !p.by_keys) issue_s(1, 0);
      release(0);
      if (kStreams == 2 && p.by_keys && n > 1) {
        ok = full(pf_k_load(1));
        if (ok) {
          tc_fence_after();
          issue_s(1, pf_k_load(1));
          release(pf_k_load(1));
        }
      }
    }
    for (int t = 0; ok && t < n; ++t) {
      if (kStreams == 2 && p.by_keys) {
        const int w = t & 1;
        ok = v_ready(t) && wait(Sm::kPFull + w, pv[w] & 1);
        if (!ok) break;
        tc_fence_after();
        issue_pv(w, pf_v_load(t, n));
        release(pf_v_load(t, n));
        if (t + 2 < n) {
          ok = full(pf_k_load(t + 2));
          if (!ok) break;
          tc_fence_after();
          issue_s(w, pf_k_load(t + 2));
          release(pf_k_load(t + 2));
        }
      } else if (kStreams == 2) {
        const bool next = t + 1 < n;
        ok = (!next || full(pf_k_load(t + 1))) && v_ready(t);
        if (!ok) break;
#pragma unroll
        for (int w = 0; w < kStreams; ++w) {
          if (w == 1 && !two) break;
          if (!wait(Sm::kPFull + w, t & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          issue_pv(w, pf_v_load(t, n));
          if (next) issue_s(w, pf_k_load(t + 1));
        }
        if (!ok) break;
        if (next) release(pf_k_load(t + 1));
        release(pf_v_load(t, n));
      } else {
        // S of tile t + 1 takes the buffer whose P the P V of tile t - 1, issued before it, read
        if (t + 1 < n) {
          ok = full(pf_k_load(t + 1));
          if (!ok) break;
          tc_fence_after();
          issue_s((t + 1) & 1, pf_k_load(t + 1));
          release(pf_k_load(t + 1));
        }
        ok = v_ready(t) && wait(Sm::kPFull + (t & 1), (t >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        issue_pv_one(t, pf_v_load(t, n));
        release(pf_v_load(t, n));
      }
    }
    // every MMA issued above completes before TMEM is released
    mma_commit_w(bar(Sm::kDrain));
    mbar_wait_drain(bar(Sm::kDrain), 0, lim);
  } else if (warp > kPfWarpMma || warp >= 4 * kStreams) {
    // ------------------------------------------------------------------ E4M3 conversion
    if constexpr (kFp8) {
      const int tid = warp > kPfWarpMma ? threadIdx.x - 32 * (kPfWarpMma + 1) : threadIdx.x;   // 4-7: 128 ..
      const int row = tid % kKeys, part = tid / kKeys;
      constexpr int kCols = D * kKeys / Sm::kConvert;   // codes of this thread: a row, or a quarter of one
      bool ok = true;
      const int loads = 2 * n;
      for (int L = 0; ok && L < loads; ++L) {
        // load L is K_0, K_1, V_0, K_2, V_1, ..., V_{n-1}
        const int tile = L == 0 ? 0 : L == loads - 1 ? n - 1 : (L & 1) ? (L + 1) / 2 : L / 2 - 1;
        ok = mbar_wait(bar(Sm::kRawFull + L % kPfRaw), (L / kPfRaw) & 1, abort, lim) &&
             mbar_wait(bar(Sm::kEmpty + L % kPfSlots), ((L / kPfSlots) & 1) ^ 1, abort, lim);
        if (!ok) break;
        const unsigned char* raw = smem + Sm::kRawAt + (L % kPfRaw) * Sm::kRawBytes;
        const uint32_t dst = base + Sm::kSlot + (L % kPfSlots) * Sm::kTileBytes;
        const bool inside = (t_begin + tile) * kKeys + row < p.len;
#pragma unroll
        for (int c = 0; c < kCols / 16; ++c) {
          const int col = part * kCols + 16 * c;   // first of 16 codes
          uint4 w = make_uint4(0u, 0u, 0u, 0u);
          if (inside) {
            const int pc = (col & 127) >> 4;
            w = *reinterpret_cast<const uint4*>(
                D >= 128 ? raw + (col >> 7) * (kKeys * 128) + row * 128 + ((pc ^ (row & 7)) << 4)
                         : raw + row * 64 + ((pc ^ ((row >> 1) & 3)) << 4));
          }
          const uint32_t at = dst + (col >> 6) * kChunkKv + row * 128;
          const int d0 = (col & 63) >> 3;   // 16-byte pieces of 8 f16
          st_shared_v4(at + ((d0 ^ (row & 7)) << 4), e4m3x2_to_f16x2(w.x), e4m3x2_to_f16x2(w.x >> 16),
                       e4m3x2_to_f16x2(w.y), e4m3x2_to_f16x2(w.y >> 16));
          st_shared_v4(at + (((d0 + 1) ^ (row & 7)) << 4), e4m3x2_to_f16x2(w.z), e4m3x2_to_f16x2(w.z >> 16),
                       e4m3x2_to_f16x2(w.w), e4m3x2_to_f16x2(w.w >> 16));
        }
        fence_proxy_async_smem();   // the MMAs read the tile through the async proxy
        mbar_arrive(bar(Sm::kRawEmpty + L % kPfRaw));
        mbar_arrive(bar(Sm::kFull + L % kPfSlots));
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax
    if (p.tile_seqs == 0) {
      // gather the Q rows, 16 bytes a thread, eight loads in flight before the first is stored
      constexpr int kPieces = D / 8, kThreads = 128 * kStreams, kStep = kThreads / kPieces, kBatch = 8;
      static_assert(kThreads % kPieces == 0 && kPieces % kBatch == 0, "Q pieces");
      const int c = threadIdx.x % kPieces;
      for (int r0 = threadIdx.x / kPieces; r0 < 128 * q_tiles; r0 += kStep * kBatch) {
        uint4 w[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int r = r0 + u * kStep;
          w[u] = make_uint4(0u, 0u, 0u, 0u);
          if (r < 128 * q_tiles && row0 + r < p.R) {
            const int b = (row0 + r) / p.rows, in = row0 + r - b * p.rows, gh = in / p.Nq;
            w[u] = *reinterpret_cast<const uint4*>(p.q + p.q_st.at(b, hkv * p.group + gh, in - gh * p.Nq) + 8 * c);
          }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int r = r0 + u * kStep, rr = r & 127;
          if (r < 128 * q_tiles)
            st_shared_v4(base + Sm::kQ + (r >> 7) * Sm::kQBytes + (c >> 3) * kChunkQ + rr * 128 + (((c & 7) ^ (rr & 7)) << 4),
                         w[u].x, w[u].y, w[u].z, w[u].w);
        }
      }
      if (!kFp8) fence_proxy_async_smem();
      mbar_arrive(bar(Sm::kQFull));
    }
    bool ok = true;
    if constexpr (kFp8) {
      // Q in place from bf16 to f16, clamped to its range: thread t takes pieces t, t + threads, ...
      ok = __all_sync(0xffffffffu, mbar_wait(bar(Sm::kQFull), 0, abort, lim));
      if (ok) {
        for (int x = threadIdx.x; x < q_tiles * int(Sm::kQBytes / 16); x += 128 * kStreams) {
          const uint32_t at = base + Sm::kQ + 16 * x;
          const uint4 w = ld_shared_v4(at);
          st_shared_v4(at, bf16x2_to_f16x2_sat_nan(w.x), bf16x2_to_f16x2_sat_nan(w.y), bf16x2_to_f16x2_sat_nan(w.z),
                       bf16x2_to_f16x2_sat_nan(w.w));
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(Sm::kQReady));
      }
    }
    const int w = warp >> 2, row = threadIdx.x & 127;
    const int mine = tiles_of(w);
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    const uint32_t s_col0 = tmem + lane_base + w * 128, o_col = tmem + lane_base + 256 + w * 128;
    const float c = p.scale_log2;
    float m = -INFINITY, l = 0.f;
    // one key tile, whose first `valid` columns are keys of the prefix
    auto step = [&](int k, int valid) -> bool {
      // the barriers of this tile's S and P, the phase that is its own, and its S
      const int at = kStreams == 2 ? w : k & 1, phase = kStreams == 2 ? k & 1 : (k >> 1) & 1;
      const uint32_t s_col = kStreams == 2 ? s_col0 : s_col0 + (k & 1) * 128;
      if (!__all_sync(0xffffffffu, mbar_wait(bar(Sm::kSFull + at), phase, abort, lim))) return false;
      tc_fence_after();
      if (valid < kKeys) {
        // the last tile: -inf over the scores past the end, in TMEM, so that one form of what follows
        // serves every tile
        for (int ch = valid / 32; ch < kKeys / 32; ++ch) {
          uint32_t r[32];
          tmem_ld32(s_col + ch * 32, r);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (32 * ch + j >= valid) r[j] = 0xff800000u;
          tmem_st32(s_col + ch * 32, r);
        }
        tmem_st_wait();
      }
      // two passes over the S columns in TMEM: the row's max, then the exponentials 32 at a time
      constexpr int kOnce = kFp8 ? 64 : kKeys;   // columns held at once
      float mx16[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) mx16[i] = -INFINITY;
#pragma unroll
      for (int from = 0; from < kKeys; from += kOnce) {
        uint32_t r[kOnce];
#pragma unroll
        for (int ch = 0; ch < kOnce / 32; ++ch) tmem_ld32_async(s_col + from + 32 * ch, r + 32 * ch);
        tmem_ld_wait();
        reg_fence<kOnce>(r);
#pragma unroll
        for (int j = 0; j < kOnce; ++j) mx16[j & 15] = fmaxf(mx16[j & 15], __uint_as_float(r[j]));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) mx16[i] = fmaxf(mx16[i], mx16[i + 8]);
      const float mx = max3f(max3f(mx16[0], mx16[1], mx16[2]), max3f(mx16[3], mx16[4], mx16[5]), fmaxf(mx16[6], mx16[7]));
      // m: the maximum, of scores (E4M3 pages, as in fa_paged_kernel) or of scores in base-2 units
      const float m_cand = fmaxf(m, kFp8 ? mx : mx * c);
      const bool grow = kFp8 ? m_cand > m && !((m_cand - m) * c <= pf_growth(true)) : m_cand > m + pf_growth(false);
      const float m_new = grow ? m_cand : m;
      const float alpha = grow ? ex2_approx(kFp8 ? (m - m_new) * c : m - m_new) : 1.f;
      const float m_use = m_new == -INFINITY ? 0.f : m_new;
      const uint64_t c2 = f2(c, c), nm2 = f2(-m_use, -m_use), lift2 = f2(kPfLift, kPfLift);
      uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
      auto exp_chunk = [&](int ch, const uint32_t* cur) {
        uint32_t pk[16];
#pragma unroll
        for (int jp = 0; jp < 16; ++jp) {
          float x0, x1;
          const uint64_t s2 = f2(__uint_as_float(cur[2 * jp]), __uint_as_float(cur[2 * jp + 1]));
          f2_split(kFp8 ? f2_fma(f2_add(s2, nm2), c2, lift2) : f2_fma(s2, c2, nm2), x0, x1);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          acc[jp & 3] = f2_add(acc[jp & 3], f2(p0, p1));
          pk[jp] = kFp8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
        }
        tmem_st16(s_col + ch * 16, pk);
      };
      {
        uint32_t ra[32], rb[32];
        tmem_ld32_async(s_col, ra);
        tmem_ld_wait();
        reg_fence<32>(ra);
#pragma unroll
        for (int ch = 0; ch < kKeys / 32; ++ch) {
          uint32_t* cur = (ch & 1) ? rb : ra;
          uint32_t* nxt = (ch & 1) ? ra : rb;
          if (ch + 1 < kKeys / 32) tmem_ld32_async(s_col + (ch + 1) * 32, nxt);
          exp_chunk(ch, cur);
          if (ch + 1 < kKeys / 32) {
            tmem_ld_wait();
            reg_fence<32>(nxt);
          }
        }
      }
      float lo, hi;
      f2_split(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), lo, hi);
      l = l * alpha + (lo + hi);
      m = m_new;
      // O may be scaled once the tile before's P V is complete: with two streams it was issued before this S
      if (kStreams == 1 && k > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar(Sm::kOFinal + 1), (k - 1) & 1, abort, lim))) return false;
        tc_fence_after();
      }
      if (k > 0 && __any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t r[32];
          tmem_ld32(o_col + ch * 32, r);
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * alpha);
          tmem_st32(o_col + ch * 32, r);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bar(Sm::kPFull + at));
      return true;
    };
    for (int k = 0; ok && k < mine; ++k) {
      const int t = t_begin + (p.by_keys && kStreams == 2 ? 2 * k + w : k);
      ok = step(k, p.len - t * kKeys);
    }
    // the partial result of this stream's rows: O / l and L
    const int R = row0 + (p.by_keys ? 0 : p.tile_rows * w) + row;
    const int part = p.by_keys && kStreams == 2 ? 2 * split + w : split;
    const long long at = ((long long)part * p.H_kv + hkv) * p.R + R;
    const bool write = (p.by_keys || w == 0 || two) && row < p.tile_rows && R < p.R;
    if (mine == 0) {
      if (write) p.l_pre[at] = -INFINITY;   // weight 0: its O is not read
    } else if (ok && __all_sync(0xffffffffu, mbar_wait(bar(Sm::kOFinal + w), 0, abort, lim))) {
      tc_fence_after();
      const float inv = l == 0.f ? 0.f : (kFp8 ? p.v_scale : 1.f) / l;
      float* dst = p.o_pre + at * D;
      // Whole 128-byte lines instead of every lane its own row: 32 columns at a time pass through 4 KB of
      // shared memory (16-byte piece c of row r at c ^ (r % 8)), from where eight lanes write a row's.
      // (Row by row the output of 256 rows took 4 us.)  In the keys form of E4M3 pages the other stream's
      // tiles may still be in the raw ring, and at d = 64 the ring is too small.
      const bool turned = !kFp8 || (D != 64 && !(p.by_keys && kStreams == 2));
      const uint32_t turn = base + Sm::kTurn + warp * 4096;
      const unsigned rows_in = __ballot_sync(0xffffffffu, write);
#pragma unroll
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t r[32];
        tmem_ld32(o_col + ch * 32, r);
        if (turned) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            st_shared_v4(turn + lane * 128 + ((j ^ (lane & 7)) << 4), __float_as_uint(__uint_as_float(r[4 * j]) * inv),
                         __float_as_uint(__uint_as_float(r[4 * j + 1]) * inv),
                         __float_as_uint(__uint_as_float(r[4 * j + 2]) * inv),
                         __float_as_uint(__uint_as_float(r[4 * j + 3]) * inv));
          __syncwarp();
          float* line = dst - lane * D + ch * 32;   // of the warp's first row
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int rr = 4 * j + (lane >> 3), c16 = lane & 7;
            const uint4 v = ld_shared_v4(turn + rr * 128 + ((c16 ^ (rr & 7)) << 4));
            if ((rows_in >> rr) & 1u) *reinterpret_cast<uint4*>(line + rr * D + 4 * c16) = v;
          }
          __syncwarp();
        } else if (write) {
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4*>(dst + ch * 32 + j) =
                make_float4(__uint_as_float(r[j]) * inv, __uint_as_float(r[j + 1]) * inv,
                            __uint_as_float(r[j + 2]) * inv, __uint_as_float(r[j + 3]) * inv);
        }
      }
      if (write)
        p.l_pre[at] = l == 0.f ? -INFINITY
                               : (kFp8 ? m * c + (lg2_approx(l) - kPfLift) : m + lg2_approx(l)) * 0.69314718055994531f;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kPfWarpTma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace fa
