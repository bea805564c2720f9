// TEST INFRASTRUCTURE ONLY: runs the paged decode kernels of paged_kernel.cuh, or the append kernel
// of append_kernel.cuh, on the host through the SIMT emulation of emu.h.
// usage: emu_paged shared  as paged, then  prefix_len splits by_keys  before the file prefix
//        emu_paged paged  B H Hkv Nq d page n_pages max_pages causal window scale fp8 ks vs warps  pk(3) pv(3)  prefix
//        emu_paged append B H Hkv N d page n_pages max_pages rot n_angles axes s0 s1 s2 s3 inter fp8 ks vs heads
//                         counts? positions?  pk(3) pv(3)  prefix
// Files prefix.q, .k, .v (pages or new rows), .table, .lengths, ...; results prefix.o, .lse or .q_out, .kp, .vp.
#include "emu.h"
#include "prefix_kernel.cuh"

#include <fstream>
#include <string>

using namespace fa;

alignas(1024) static unsigned char dec_smem[232448];

template <class T>
std::vector<T> read_all(const std::string& path) {
  std::ifstream f(path, std::ios::binary | std::ios::ate);
  if (!f) { std::fprintf(stderr, "no %s\n", path.c_str()); std::exit(2); }
  std::vector<T> v(size_t(f.tellg()) / sizeof(T));
  f.seekg(0);
  f.read(reinterpret_cast<char*>(v.data()), v.size() * sizeof(T));
  return v;
}
template <class T>
void write_file(const std::string& path, const std::vector<T>& v) {
  std::ofstream f(path, std::ios::binary);
  f.write(reinterpret_cast<const char*>(v.data()), v.size() * sizeof(T));
}

// With "hidden" in front of the arguments: before every grid, what other grids or the host have written
// is replaced by other values, and comes back when a thread of the grid waits for the grids before.
struct Hidden {
  unsigned char* at;
  std::vector<unsigned char> kept;
  int fill;
};
static bool hide_inputs = false;
// With "second" there the paged grid's CTA 1 goes first, and CTA 0 last: it may be taken over.
static unsigned first_cta = 0;
static std::vector<Hidden> hidden;
static bool is_hidden = false;
static std::mutex hidden_mu;
template <class T>
static void hideable(std::vector<T>& v, int fill) {
  if (!v.empty()) hidden.push_back(Hidden{reinterpret_cast<unsigned char*>(v.data()), std::vector<unsigned char>(v.size() * sizeof(T)), fill});
}
static void hide() {
  if (!hide_inputs) return;
  for (Hidden& h : hidden) {
    std::copy(h.at, h.at + h.kept.size(), h.kept.begin());
    std::memset(h.at, h.fill, h.kept.size());
  }
  is_hidden = true;
  emu_on_dep_wait = [] {
    std::lock_guard<std::mutex> lk(hidden_mu);
    if (!is_hidden) return;
    for (Hidden& h : hidden) std::copy(h.kept.begin(), h.kept.end(), h.at);
    is_hidden = false;
  };
}

static char** arg;
static int num() { return atoi(*arg++); }
static float fnum() { return float(atof(*arg++)); }
static Strides strides3() {
  Strides s;
  s.b = atoll(*arg++);
  s.h = atoll(*arg++);
  s.n = atoll(*arg++);
  return s;
}
static Strides packed(int heads, int N, int d) { return Strides{(long long)heads * N * d, (long long)N * d, d}; }

// q in boxes of a tile's whole sequences, as fa_fwd_shared encodes it
static CUtensorMap q_map(const PrefixParams& x, int d) {
  CUtensorMap m = {};
  m.base = reinterpret_cast<const unsigned char*>(x.q);
  m.dims[0] = uint64_t(d); m.dims[1] = uint64_t(x.Nq); m.dims[2] = uint64_t(x.H_kv) * x.group; m.dims[3] = uint64_t(x.R / x.rows);
  m.strides[0] = uint64_t(x.q_st.n) * 2; m.strides[1] = uint64_t(x.q_st.h) * 2; m.strides[2] = uint64_t(x.q_st.b) * 2;
  m.box_x = 64;
  m.box_rows = uint32_t(x.Nq);
  m.box_heads = uint32_t(x.group);
  m.box_batch = uint32_t(x.tile_seqs);
  m.esize = 2;
  m.swizzle = 128;
  return m;
}

template <int D, bool kFp8>
void run_paged(const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p, const PrefixParams* x) {
  if (x) {
    CUtensorMap pk = tk, pv = tv;
    pk.box_rows = pv.box_rows = uint32_t(x->box_rows);
    hide();
    emu_launch(unsigned(x->H_kv * x->n_splits * x->row_groups), pf_threads(kFp8), PrefixSmem<D, kFp8>::kAlloc,
               [&] { fa_prefix_kernel<D, kFp8>(q_map(*x, D), pk, pv, *x); }, dec_smem);
  }
  hide();
  emu_first_cta = first_cta;
  emu_launch(unsigned(p.warps) * pg_parts(D), 32, PgLayout<D, kFp8>::kSmemBytes,
             [&] { fa_paged_kernel<D, kFp8>(tk, tv, p); }, dec_smem);
  emu_first_cta = 0;
  hide();
  // four warps a row, or one when there are many rows
  emu_launch(unsigned(p.total_rows), p.total_rows <= 48 ? 32 * kPgMergeWarps : 32, pg_merge_smem(D),
             [&] { fa_paged_merge_kernel<D, PgLayout<D, kFp8>::kStep>(p); }, dec_smem);
}

static int paged_main(bool shared) {
  const int B = num(), H = num(), Hkv = num(), Nq = num(), d = num(), page = num(), n_pages = num(), max_pages = num(),
            causal = num(), window = num();
  const float scale = fnum();
  const bool fp8 = num();
  const float k_scale = fnum(), v_scale = fnum();
  const int warps = num();
  const Strides ks = strides3(), vs = strides3();
  const int prefix_len = shared ? num() : 0, splits = shared ? num() : 0, by_keys = shared ? num() : 0;
  const std::string prefix = *arg++;
  auto q = read_all<uint16_t>(prefix + ".q");
  auto k = read_all<unsigned char>(prefix + ".k"), v = read_all<unsigned char>(prefix + ".v");
  auto table = read_all<int>(prefix + ".table"), lengths = read_all<int>(prefix + ".lengths");
  std::vector<int> counts;   // a file of the ragged calls alone
  if (std::ifstream(prefix + ".counts")) counts = read_all<int>(prefix + ".counts");
  std::vector<uint16_t> o(q.size(), 0x7fc0);
  std::vector<float> lse(size_t(B) * H * Nq, NAN);
  PagedParams p = {};
  const int part_rows = std::min(H / Hkv * Nq, kDecRows);
  std::vector<float> o_part(size_t(2) * warps * pg_parts(d) * part_rows * d, NAN), l_part(o_part.size() / d, NAN);
  p.part_rows = part_rows;
  p.q = reinterpret_cast<const __nv_bfloat16*>(q.data());
  p.o = reinterpret_cast<__nv_bfloat16*>(o.data());
  p.lse = lse.data();
  p.o_part = o_part.data();
  p.l_part = l_part.data();
  p.table = table.data();
  p.table_stride = max_pages;
  p.lengths = lengths.data();
  p.counts = counts.empty() ? nullptr : counts.data();
  p.q_st = p.o_st = packed(H, Nq, d);
  p.total_rows = (long long)B * H * Nq;
  p.B = B; p.H = H; p.H_kv = Hkv; p.group = H / Hkv; p.Nq = Nq;
  p.rows = p.group * Nq;
  p.row_blocks = (p.rows + kDecRows - 1) / kDecRows;
  p.n_pages = n_pages; p.page_size = page; p.max_pages = max_pages;
  p.causal = causal; p.window = window; p.warps = warps;
  p.scale_log2 = scale * (fp8 ? k_scale : 1.f) * 1.4426950408889634f;
  p.v_scale = v_scale;
  p.wait_limit_ns = 60000000000ull;   // (a loaded host runs the emulated threads late)
  auto kv_map = [&](const void* base, const Strides& s) {
    CUtensorMap m;
    const uint32_t es = fp8 ? 1 : 2;
    m.base = static_cast<const unsigned char*>(base);
    m.dims[0] = uint64_t(d); m.dims[1] = uint64_t(page); m.dims[2] = uint64_t(Hkv); m.dims[3] = uint64_t(n_pages);
    m.strides[0] = uint64_t(s.n) * es; m.strides[1] = uint64_t(s.h) * es; m.strides[2] = uint64_t(s.b) * es;
    m.box_x = fp8 && d >= 128 ? 128 : 64;
    m.box_rows = kDecKeys;
    m.esize = es;
    m.swizzle = fp8 && d < 128 ? 64 : 128;
    return m;
  };
  const CUtensorMap tk = kv_map(k.data(), ks), tv = kv_map(v.data(), vs);
  PrefixParams x = {};
  std::vector<int> pages;
  std::vector<float> o_row, l_row, o_pre, l_pre;
  if (shared) {
    pages = read_all<int>(prefix + ".pages");
    x.q = p.q;
    x.pages = pages.data();
    x.q_st = p.q_st;
    x.R = B * p.rows; x.rows = p.rows; x.Nq = Nq; x.group = p.group; x.H_kv = Hkv;
    x.len = prefix_len; x.n_pages = n_pages; x.page_size = page;
    x.box_rows = 16;
    while (x.box_rows * 2 <= pf_keys(d) && page % (x.box_rows * 2) == 0) x.box_rows *= 2;
    x.n_tiles = (prefix_len + pf_keys(d) - 1) / pf_keys(d);
    x.tiles_per_split = (x.n_tiles + splits - 1) / splits;
    x.n_splits = (x.n_tiles + x.tiles_per_split - 1) / x.tiles_per_split;
    x.by_keys = by_keys;
    x.tile_seqs = std::min(B, 128 / p.rows);
    x.tile_rows = x.tile_seqs ? x.tile_seqs * p.rows : 128;
    const int per = x.tile_rows * (by_keys ? 1 : pf_streams(d));
    x.row_groups = (x.R + per - 1) / per;
    x.scale_log2 = p.scale_log2;
    x.v_scale = v_scale;
    x.wait_limit_ns = 60000000000ull;
    p.n_pre = x.n_splits * (by_keys ? 2 : 1);
    o_row.assign(size_t(p.total_rows) * d, NAN);
    l_row.assign(size_t(p.total_rows), NAN);
    o_pre.assign(size_t(p.n_pre) * p.total_rows * d, NAN);
    l_pre.assign(size_t(p.n_pre) * p.total_rows, NAN);
    p.o_row = o_row.data();
    p.l_row = l_row.data();
    p.o_pre = x.o_pre = o_pre.data();
    p.l_pre = x.l_pre = l_pre.data();
  }
  hideable(q, 0x7f);
  hideable(k, 0);
  hideable(v, 0);
  hideable(table, 0);
  hideable(lengths, 0);
  hideable(counts, 0);
  for (auto* part : {&o_part, &l_part, &o_row, &l_row, &o_pre, &l_pre}) hideable(*part, 0xff);
  if (shared) hideable(pages, 0);
  const PrefixParams* xp = shared ? &x : nullptr;
  if (d == 64) fp8 ? run_paged<64, true>(tk, tv, p, xp) : run_paged<64, false>(tk, tv, p, xp);
  else if (d == 128) fp8 ? run_paged<128, true>(tk, tv, p, xp) : run_paged<128, false>(tk, tv, p, xp);
  else fp8 ? run_paged<256, true>(tk, tv, p, xp) : run_paged<256, false>(tk, tv, p, xp);
  write_file(prefix + ".o", o);
  write_file(prefix + ".lse", lse);
  std::printf("status %d\n", g_status);
  return 0;
}

template <int D, bool kFp8, bool kInter, bool kOneAxis, int kHeads>
void run_append(AppendParams p) {
  p.q_groups = (p.H + kHeads - 1) / kHeads;
  p.kv_groups = (p.H_kv + kHeads - 1) / kHeads;
  const int per_token = (p.q_groups + 2 * p.kv_groups) * (D / 16);
  p.tokens_per_block = per_token >= kAppThreads ? 1 : kAppThreads / per_token;
  const unsigned gx = unsigned((p.tokens - 1) / p.tokens_per_block + 1);
  const unsigned gy = unsigned((p.tokens_per_block * per_token + kAppThreads - 1) / kAppThreads);
  for (unsigned y = 0; y < gy; ++y)
    emu_launch(gx, kAppThreads, 0, [&] {
      blockIdx.y = y;
      fa_append_kernel<D, kFp8, kInter, kOneAxis, kHeads>(p);
    });
}
template <int D, bool kFp8, bool kInter>
void run_append_h(const AppendParams& p, int heads) {
  if (p.axes > 1) heads == 1 ? run_append<D, kFp8, kInter, false, 1>(p) : run_append<D, kFp8, kInter, false, 4>(p);
  else heads == 1 ? run_append<D, kFp8, kInter, true, 1>(p) : run_append<D, kFp8, kInter, true, 4>(p);
}
template <int D>
void run_append_d(const AppendParams& p, bool fp8, bool inter, int heads) {
  if (fp8) inter ? run_append_h<D, true, true>(p, heads) : run_append_h<D, true, false>(p, heads);
  else inter ? run_append_h<D, false, true>(p, heads) : run_append_h<D, false, false>(p, heads);
}

static int append_main() {
  AppendParams p = {};
  p.B = num(); p.H = num(); p.H_kv = num(); p.N = num();
  const int d = num();
  p.page_size = num(); p.n_pages = num(); p.max_pages = num();
  p.rot = num(); p.n_angles = num(); p.axes = num();
  int at = 0;
  for (int a = 0; a < 4; ++a) p.edge[a] = at += num();
  const bool inter = num(), fp8 = num();
  const float ks = fnum(), vs = fnum();
  const int heads = num(), with_counts = num(), with_positions = num();
  p.kp_st = strides3();
  p.vp_st = strides3();
  const std::string prefix = *arg++;
  auto q = read_all<uint16_t>(prefix + ".q"), k = read_all<uint16_t>(prefix + ".k"), v = read_all<uint16_t>(prefix + ".v");
  auto kp = read_all<unsigned char>(prefix + ".kp"), vp = read_all<unsigned char>(prefix + ".vp");
  auto table = read_all<int>(prefix + ".table"), lengths = read_all<int>(prefix + ".lengths");
  std::vector<int> counts, positions;
  if (with_counts) counts = read_all<int>(prefix + ".counts");
  if (with_positions) positions = read_all<int>(prefix + ".positions");
  auto cos_t = read_all<float>(prefix + ".cos"), sin_t = read_all<float>(prefix + ".sin");
  std::vector<uint16_t> q_out(q.size(), 0x4242);
  p.q = reinterpret_cast<const __nv_bfloat16*>(q.data());
  p.k = reinterpret_cast<const __nv_bfloat16*>(k.data());
  p.v = reinterpret_cast<const __nv_bfloat16*>(v.data());
  p.q_out = reinterpret_cast<__nv_bfloat16*>(q_out.data());
  p.k_pages = kp.data();
  p.v_pages = vp.data();
  p.q_st = p.qo_st = packed(p.H, p.N, d);
  p.k_st = p.v_st = packed(p.H_kv, p.N, d);
  p.table = table.data();
  p.table_stride = p.max_pages;
  p.lengths = lengths.data();
  p.counts = with_counts ? counts.data() : nullptr;
  p.positions = with_positions ? positions.data() : nullptr;
  p.cos_t = cos_t.data();
  p.sin_t = sin_t.data();
  p.tokens = p.B * p.N;
  p.k_inv = 1.f / ks;
  p.v_inv = 1.f / vs;
  if (d == 64) run_append_d<64>(p, fp8, inter, heads);
  else if (d == 128) run_append_d<128>(p, fp8, inter, heads);
  else run_append_d<256>(p, fp8, inter, heads);
  write_file(prefix + ".q_out", q_out);
  write_file(prefix + ".kp", kp);
  write_file(prefix + ".vp", vp);
  std::printf("status %d\n", g_status);
  return 0;
}

int main(int argc, char** argv) {
  if (argc < 2) return 2;
  hide_inputs = std::string(argv[1]) == "hidden";
  first_cta = std::string(argv[1]) == "second";
  arg = argv + (hide_inputs || first_cta ? 3 : 2);
  if (arg > argv + argc) return 2;
  const std::string what = arg[-1];
  return what == "append" ? append_main() : paged_main(what == "shared");
}
