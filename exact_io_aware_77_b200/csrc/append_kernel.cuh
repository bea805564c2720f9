// Appending new rows to a paged key/value cache, with the position rotation applied on the way.
//
// Element pair p of a head, (a, b), standing at position t of the pair's axis becomes
//   a' = a cos(t, p) - b sin(t, p),   b' = b cos(t, p) + a sin(t, p),
// with cos and sin read from the caller's fp32 tables [n_angles, rot / 2] and the arithmetic in
// fp32.  The rotated q goes back as bf16, the rotated k and the plain v into the sequence's pages,
// rounded once, to bf16 or to E4M3 codes of value / scale.
//
// The work is reading and writing each row once.  A thread owns 16 elements of a head row of one
// token: 8 pairs, as two 16-byte pieces rot / 2 apart (or adjacent, for interleaved pairs), of
// kHeads neighbouring heads of q, k or v at a time, so that its angles and addresses serve all of
// them and the heads' loads are in flight together.  A row's page is looked up by every
// thread that writes to it: the lookups of a warp hit the same few words.  HBM bounds it: 8192 tokens of
// 32 + 8 + 8 heads of 128 (206 MB) take 38.7 us, 5.3 TB/s; one token each of eight sequences takes 6 us
// from a cold start, all latency.  4444 padded rows with three axes into E4M3 pages (68 MB) take 18.3 us: a
// thread's loads depend on one another four deep (count and length, rows, positions and page, angles), and 80
// registers leave three CTAs an SM to hide that.
#pragma once

#include <cstdint>

#include "decode_ops.cuh"
#include "fp8_ops.cuh"
#include "sm100.cuh"

namespace fa {

constexpr int FA_DEVICE_BAD_INDEX = 4;   // device status bit: a page, length, count or position out of range

constexpr int kAppThreads = 256;
constexpr int kAppMaxAxes = 4;

struct AppendParams {
  const __nv_bfloat16* q;       // [B, H, N, d]; H = 0 without q
  const __nv_bfloat16* k;       // [B, H_kv, N, d]
  const __nv_bfloat16* v;
  __nv_bfloat16* q_out;
  void* k_pages;                // [n_pages, H_kv, page_size, d], bf16 or E4M3 codes
  void* v_pages;
  Strides q_st, k_st, v_st, qo_st, kp_st, vp_st;   // pages: b = page stride
  const int* table;             // [B, max_pages], rows table_stride apart
  const int* lengths;           // [B] keys held after the append
  const int* counts;            // [B] valid rows, or nullptr: all N
  const int* positions;         // [axes, B, N], or nullptr: the row's slot
  const float* cos_t;           // [n_angles, rot / 2]; rot = 0: no rotation
  const float* sin_t;
  long long table_stride;
  int tokens;                   // B * N
  int B, N, H, H_kv;
  int n_pages, page_size, max_pages;
  int rot, n_angles, axes;
  int edge[kAppMaxAxes];        // first pair past each axis
  float k_inv, v_inv;           // E4M3: codes hold value * inv
  int q_groups, kv_groups;      // groups of kHeads heads of q, and of k or v
  int tokens_per_block;
};

__device__ __forceinline__ float app_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float app_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 8 bf16 as fp32
__device__ __forceinline__ void app_unpack(const uint4& w, float* f) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = app_lo(x[i]);
    f[2 * i + 1] = app_hi(x[i]);
  }
}
__device__ __forceinline__ uint4 app_pack_bf16(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ uint2 app_pack_e4m3(const float* f, float inv) {
  uint2 w;
  w.x = f32x2_to_e4m3x2(f[0] * inv, f[1] * inv) | (f32x2_to_e4m3x2(f[2] * inv, f[3] * inv) << 16);
  w.y = f32x2_to_e4m3x2(f[4] * inv, f[5] * inv) | (f32x2_to_e4m3x2(f[6] * inv, f[7] * inv) << 16);
  return w;
}

// The angles of pairs p0 .. p0 + 7 of a row at these positions of its axes, which lie within the tables:
// one load of four where they share an axis.
template <bool kOneAxis>
__device__ __forceinline__ void app_angles(const AppendParams& p, const int* pos, int p0, float* cs, float* sn) {
  const int half = p.rot >> 1;
  auto load4 = [&](int pos, int q0) {
    const long long at = (long long)pos * half + q0;
    const float4 fc = *reinterpret_cast<const float4*>(p.cos_t + at);
    const float4 fs = *reinterpret_cast<const float4*>(p.sin_t + at);
    float* c = cs + (q0 - p0);
    float* s = sn + (q0 - p0);
    c[0] = fc.x, c[1] = fc.y, c[2] = fc.z, c[3] = fc.w;
    s[0] = fs.x, s[1] = fs.y, s[2] = fs.z, s[3] = fs.w;
  };
  if constexpr (kOneAxis) {
    load4(pos[0], p0);
    load4(pos[0], p0 + 4);
  } else {
    auto axis_of = [&](int pair) {
      int x = 0;
#pragma unroll
      for (int a = 1; a < kAppMaxAxes; ++a)
        if (a < p.axes && pair >= p.edge[a - 1]) x = a;
      return x;
    };
    auto pos_of = [&](int axis) { return axis == 0 ? pos[0] : axis == 1 ? pos[1] : axis == 2 ? pos[2] : pos[3]; };
#pragma unroll
    for (int g = 0; g < 8; g += 4) {
      const int q0 = p0 + g, first = axis_of(q0);
      if (first == axis_of(q0 + 3)) {
        load4(pos_of(first), q0);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const long long at = (long long)pos_of(axis_of(q0 + e)) * half + q0 + e;
          cs[g + e] = p.cos_t[at];
          sn[g + e] = p.sin_t[at];
        }
      }
    }
  }
}

// kInter: pairs (2p, 2p + 1); otherwise (p, p + rot / 2).  kOneAxis: every pair turns by one position.
template <int D, bool kFp8, bool kInter, bool kOneAxis, int kHeads>
__global__ void __launch_bounds__(kAppThreads) fa_append_kernel(const AppendParams p) {
  constexpr int kChunks = D / 16;
  // this grid may be scheduled while the one before it runs (q, k and v's producer, or a reader of
  // the cache); the next one, while this one does
  grid_dep_launch_dependents();
  grid_dep_wait();
  const int groups = p.q_groups + 2 * p.kv_groups;
  const int item = int(blockIdx.y) * kAppThreads + int(threadIdx.x);
  const int t_in = item / (groups * kChunks);
  const int token = int(blockIdx.x) * p.tokens_per_block + t_in;
  if (t_in >= p.tokens_per_block || token >= p.tokens) return;
  const int rest = item - t_in * (groups * kChunks);
  int hg = rest / kChunks;
  const int c = rest % kChunks;
  const int b = token / p.N, i = token - b * p.N;
  const int said = p.counts ? p.counts[b] : p.N;
  const int count = min(max(said, 0), p.N);
  if (said != count) atomicOr(&g_status, FA_DEVICE_BAD_INDEX);
  const int slot = max(p.lengths[b], 0) - count + i;
  if (i >= count || slot < 0) return;   // padding: the row has no place, nothing of it is written

  // q, k or v; its heads h0 .. h0 + n - 1 are this thread's
  const int what = hg < p.q_groups ? 0 : hg < p.q_groups + p.kv_groups ? 1 : 2;
  hg -= what == 0 ? 0 : what == 1 ? p.q_groups : p.q_groups + p.kv_groups;
  const int h0 = hg * kHeads, n = min(kHeads, (what == 0 ? p.H : p.H_kv) - h0);
  const Strides st = what == 0 ? p.q_st : what == 1 ? p.k_st : p.v_st;
  const __nv_bfloat16* src = (what == 0 ? p.q : what == 1 ? p.k : p.v) + st.at(b, h0, i);
  // this thread's two 8-element pieces, rotated or not
  const bool turn = 16 * c < p.rot && what != 2;
  const bool apart = 16 * c < p.rot && !kInter;
  const int e0 = apart ? 8 * c : 16 * c, e1 = apart ? (p.rot >> 1) + 8 * c : 16 * c + 8;
  uint4 x0[kHeads], x1[kHeads];   // the heads' loads first: they wait for the padding test alone
#pragma unroll
  for (int j = 0; j < kHeads; ++j)
    if (j < n) {
      x0[j] = *reinterpret_cast<const uint4*>(src + j * st.h + e0);
      x1[j] = *reinterpret_cast<const uint4*>(src + j * st.h + e1);
    }

  // A row is stored whole or not at all, so every thread of it looks at the positions of all its axes.
  int pos[kOneAxis ? 1 : kAppMaxAxes];
#pragma unroll
  for (int a = 0; a < (kOneAxis ? 1 : kAppMaxAxes); ++a) {
    pos[a] = 0;
    if (a < p.axes) pos[a] = p.positions ? p.positions[(long long)a * p.tokens + token] : slot;
  }

  // place of the rows: q_out, or the sequence's page
  Strides to = p.qo_st;
  long long at = to.at(b, h0, i);
  if (what != 0) {
    const int pg = slot / p.page_size;
    const int page = pg < p.max_pages ? p.table[(long long)b * p.table_stride + pg] : -1;
    if (unsigned(page) >= unsigned(p.n_pages)) {
      atomicOr(&g_status, FA_DEVICE_BAD_INDEX);
      return;
    }
    to = what == 1 ? p.kp_st : p.vp_st;
    at = to.at(page, h0, slot - pg * p.page_size);
  }

  bool in_tables = true;
#pragma unroll
  for (int a = 0; a < (kOneAxis ? 1 : kAppMaxAxes); ++a)
    if (a < p.axes) in_tables = in_tables && unsigned(pos[a]) < unsigned(p.n_angles);
  if (!in_tables) {
    atomicOr(&g_status, FA_DEVICE_BAD_INDEX);
    return;
  }

  float cs[8], sn[8];
  if (turn) app_angles<kOneAxis>(p, pos, 8 * c, cs, sn);

  const bool codes = kFp8 && what != 0;
  const float inv = what == 1 ? p.k_inv : p.v_inv;
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    if (j >= n) break;
    uint4 y0 = x0[j], y1 = x1[j];   // elements that stay bf16 unrotated keep their bits
    if (turn || codes) {
      float f[16];
      app_unpack(x0[j], f);
      app_unpack(x1[j], f + 8);
      if (turn) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float& a = kInter ? f[2 * e] : f[e];
          float& w = kInter ? f[2 * e + 1] : f[8 + e];
          const float ra = a * cs[e] - w * sn[e], rw = w * cs[e] + a * sn[e];
          a = ra;
          w = rw;
        }
      }
      if (codes) {
        uint8_t* dst = static_cast<uint8_t*>(what == 1 ? p.k_pages : p.v_pages) + at + j * to.h;
        *reinterpret_cast<uint2*>(dst + e0) = app_pack_e4m3(f, inv);
        *reinterpret_cast<uint2*>(dst + e1) = app_pack_e4m3(f + 8, inv);
        continue;
      }
      y0 = app_pack_bf16(f);
      y1 = app_pack_bf16(f + 8);
    }
    __nv_bfloat16* dst = (what == 0 ? p.q_out : static_cast<__nv_bfloat16*>(what == 1 ? p.k_pages : p.v_pages)) + at + j * to.h;
    *reinterpret_cast<uint4*>(dst + e0) = y0;
    *reinterpret_cast<uint4*>(dst + e1) = y1;
  }
}

}  // namespace fa
