// msa_dense.cu — causal GQA attention over the whole paged NVFP4 cache (msa_dense_attn).
//
// o = softmax(scale q K^T) V over all keys up to each query's position, K and V dequantised to
// E4M3. The work is a list of units (query tile, group, key block): a tile is up to 8 query tokens
// of one sequence (16 where sequences may hold more than 8), its 16 heads a token the rows of the
// MMAs' M = 128; a unit is one 128-key block of one group's K and V. Units are numbered sequence by
// sequence, tile by tile, group by group, and cut into equal spans of kTunedSms CTAs, so that every
// SM streams the same number of blocks whatever the lengths (blocks cost the same where all tiles have one form;
// a tile of more than 8 tokens costs more a block than one of fewer); a (tile, group) cut by a span's border
// leaves its parts' unnormalised sums in the workspace and a second kernel joins them, in order.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <math_constants.h>
#include <stdint.h>

#include <type_traits>

#include "msa.h"
#include "msa_attn_tile.cuh"
#include "msa_device.cuh"
#include "msa_host.h"

namespace msa {
namespace {

constexpr int kSpans = msa_host::kTunedSms;  // CTAs
constexpr int kRows = 128;                   // rows of one MMA tile: 8 tokens x 16 heads
constexpr int kTileTok = kRows / kHPG;       // 8

struct DenseParams {
  int32_t B, T, maxb, max_q_len, num_pages, tile_tok, tile_log2;  // tokens a tile: 1, 8 or 16
  const int32_t *qsl, *seq_lens, *block_table;
  float scale_log2;
  uint16_t* out;
  float* lse;
  uint32_t* status;
  int4* rec;       // [kSpans] the cut (tile, group) that starts in span c: parts, t0, tokens, group
  float* part_o;   // [kSpans][2][tile rows][128] unnormalised sums
  float2* part_ml; // [kSpans][2][tile rows] reference maximum (log2) and sum
};

// ------------------------------------------------------------------ units -------------
// Sequence b's share: its query tokens and cache length, or none (zero tokens, or a row that is
// not consistent).
struct Seq {
  int q0, ql, L;
};
__device__ __forceinline__ Seq load_seq(const DenseParams& p, int b, bool* bad) {
  Seq s;
  s.q0 = p.qsl[b];
  s.ql = p.qsl[b + 1] - s.q0;
  s.L = p.seq_lens[b];
  *bad = s.q0 < 0 || s.ql < 0 || s.q0 > p.T - s.ql || s.ql > p.max_q_len || s.L < s.ql ||
         static_cast<int64_t>(s.L) > static_cast<int64_t>(p.maxb) * kBS;
  if (*bad && s.ql == 0) *bad = false;  // a padded row: skipped, whatever it says
  if (*bad || s.ql < 0) s.ql = 0;
  return s;
}

// sum_{j < n} floor(j / 2^r)
__device__ __forceinline__ int64_t floor_sum(int64_t n, int r) {
  const int64_t m = n >> r;
  return ((m * (m - 1) / 2) << r) + (n - (m << r)) * m;
}
// Key blocks of tiles 0 .. k - 1 of a sequence, all full (2^t tokens): tile i ends at position
// L - ql + 2^t (i + 1) - 1.
__device__ __forceinline__ int64_t tile_blocks(const Seq& s, int t, int64_t k) {
  const int64_t a = (static_cast<int64_t>(s.L) - s.ql + (1 << t) - 1) >> t;
  return k + floor_sum(a + k, 7 - t) - floor_sum(a, 7 - t);
}
__device__ __forceinline__ int tiles_of(const Seq& s, int t) { return (s.ql + (1 << t) - 1) >> t; }
__device__ __forceinline__ int64_t seq_units(const Seq& s, int t) {
  if (s.ql == 0) return 0;
  return kGroups * (tile_blocks(s, t, tiles_of(s, t) - 1) + (s.L - 1) / kBS + 1);
}

// Where a span starts: sequence, tile, group, block; its first unit's number and count; all units.
struct Start {
  int64_t first, count, total;
  Seq seq;
  int b, tile, g, j, pad;
};

// One (tile, group) of a span, or part of it.
struct Seg {
  int32_t n;       // blocks here (-1: the end of the list)
  int32_t j0;      // the first
  int32_t t0, ntok, p0, g;  // first token, tokens, the first one's position, group
  int32_t part;    // -1: the whole (tile, group); else its place in the workspace (0 or 1)
  int32_t bad;     // first key position of the segment on a bad page (2^31 - 1: none)
  int32_t cut;     // V counts before this key of the segment: up to the last position, or a bad page
};

// ------------------------------------------------------------------ the kernel --------
constexpr int kStageBytes = 2 * kRegion;       // 18,432: a head's K and V rows of a page
constexpr int kKTile = kBS * kD;               // E4M3
constexpr int kVTile = 2 * kBS * kD;           // f16
constexpr int kVLbo = kVTile / 2, kVSbo = 1024;  // MN-major: 64-dim halves, 8-key groups
constexpr int kSegs = 4;
constexpr int kWarpProd = 0, kWarpS = 1, kWarpPv = 2, kWarpDq = 4, kWarpSm = 12;
constexpr int kWarps = 20, kThreads = 32 * kWarps;
constexpr int kSegUsers = 1 + 1 + 8 + 8;
constexpr uint32_t kTmemCols = 512, kColO = 256;
constexpr int kHalf = kBS / 2;                   // keys of one step of a slot
// P = 2^(z - max + kRaise) where the reference is set, and a row keeps it while the sum of P over a
// step's 64 keys stays within kMostSum, inside f16 (65,504). f16 rounds a P by at least 2^-25: 2^-28 of the largest, so
// that keys far below one that they outweigh together keep their weight. (With 5, a prompt's rows move
// their references more often: 32 x 16K of 8 tokens 122.4 us, 120.3 with 3.)
constexpr float kRaise = 3.0f, kMostSum = 61440.0f;
constexpr std::integral_constant<int, 0> kX0{};
constexpr std::integral_constant<int, 1> kX1{};

struct Smem {
  static constexpr int kStages = 5;            // raw K + V regions in flight
  static constexpr int kQTile = kRows * kD;    // 16 KB
  static constexpr size_t kOffStage = 0;
  static constexpr size_t kOffQ = kOffStage + kStages * static_cast<size_t>(kStageBytes);
  static constexpr size_t kOffK = kOffQ + 2 * static_cast<size_t>(kQTile);
  static constexpr size_t kOffV = kOffK + 2 * static_cast<size_t>(kKTile);
  static constexpr size_t kOffLut = kOffV + 2 * static_cast<size_t>(kVTile);
  static constexpr size_t kOffMl = kOffLut + 256 * 8;                    // [2][2][128] float2
  static constexpr size_t kOffSeg = kOffMl + 2 * 2 * kRows * 8;
  static constexpr size_t kOffStart = kOffSeg + kSegs * sizeof(Seg);
  static constexpr size_t kOffScan = kOffStart + sizeof(Start);          // [kWarps] int64
  static constexpr size_t kOffBar = kOffScan + kWarps * 8;
  static constexpr int kNumBars = 2 * kSegs + 2 * kStages + 28;
  static constexpr size_t kOffMisc = kOffBar + 8 * kNumBars;
  static constexpr size_t kBytes = 1024 + kOffMisc + 16;
};
static_assert(kStageBytes % 1024 == 0 && Smem::kOffQ % 1024 == 0 && Smem::kOffK % 1024 == 0 && Smem::kOffV % 1024 == 0,
              "swizzled tiles start on 1024-B boundaries");
static_assert(Smem::kOffStart % 8 == 0 && Smem::kOffBar % 8 == 0 && Smem::kBytes <= 232448, "shared memory per CTA");

struct Bars {
  uint64_t *seg_full, *seg_empty, *raw_full, *raw_empty, *q_full, *q_empty, *k_full, *k_empty, *v_full, *v_empty,
      *s_full, *p_full, *pv_done, *o_free, *ml, *fin;
  __device__ explicit Bars(uint8_t* smem) {
    uint64_t* b = reinterpret_cast<uint64_t*>(smem + Smem::kOffBar);
    seg_full = b;
    seg_empty = b + kSegs;
    b += 2 * kSegs;
    raw_full = b;
    raw_empty = b + Smem::kStages;
    b += 2 * Smem::kStages;
    q_full = b;
    q_empty = b + 2;
    k_full = b + 4;
    k_empty = b + 6;
    v_full = b + 8;
    v_empty = b + 10;
    s_full = b + 12;   // [slot][half], as p_full and pv_done
    p_full = b + 16;
    pv_done = b + 20;
    o_free = b + 24;
    ml = b + 25;
    fin = b + 26;  // [0] the S issuer, [1] the PV issuer
    static_assert(Smem::kNumBars == 2 * kSegs + 2 * Smem::kStages + 28, "barrier area");
  }
};

// The sum of the units of all sequences, this span's share of them and where it starts: every
// thread of the CTA takes a run of sequences, a scan over the threads gives each run its first unit.
__device__ __forceinline__ void find_start(const DenseParams& p, Start* st, int64_t* scan, int threads) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = p.B <= threads ? 1 : (p.B + threads - 1) / threads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  int64_t mine = 0;
  bool any_bad = false;
  Seq one{};  // the run's sequence where there is one a thread (not read again)
  for (int b = b0; b < b1; ++b) {
    bool bad;
    one = load_seq(p, b, &bad);
    mine += seq_units(one, p.tile_log2);
    any_bad |= bad;
  }
  if (any_bad && blockIdx.x == 0) set_status(p.status, MSA_ERR_INVALID_ARG);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
  const int holding = (p.B + 32 * per - 1) / (32 * per);  // warps that hold sequences
  for (int w = 0; w < holding; ++w) {
    const int64_t v = scan[w];
    if (w < warp) before += v;
    total += v;
  }
  // span c: units c total / kSpans .. ; one unit each where there are fewer (no span but the last ones is empty)
  const int64_t first = total < kSpans ? min(static_cast<int64_t>(blockIdx.x), total) : blockIdx.x * total / kSpans;
  const int64_t end = total < kSpans ? min(first + 1, total) : (blockIdx.x + 1) * total / kSpans;
  if (tid == 0) {
    st->first = first;
    st->count = end - first;
    st->total = total;
  }
  int64_t at = before + incl - mine;  // the first unit of this thread's run
  if (end > first && first >= at && first < at + mine) {
    for (int b = b0; b < b1; ++b) {
      bool bad;
      const Seq s = per == 1 ? one : load_seq(p, b, &bad);
      const int64_t u = per == 1 ? mine : seq_units(s, p.tile_log2);
      if (first < at + u) {
        const int64_t rel = first - at;
        int lo = 0, hi = tiles_of(s, p.tile_log2) - 1;  // the last tile that starts at or before it
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (kGroups * tile_blocks(s, p.tile_log2, mid) <= rel) lo = mid; else hi = mid - 1;
        }
        int in = static_cast<int>(rel - kGroups * tile_blocks(s, p.tile_log2, lo)), g = 0;  // < 4 nb
        const int last = min((lo + 1) << p.tile_log2, s.ql) - 1;  // the tile's last token
        const int nb = (s.L - s.ql + last) / kBS + 1;
        while (in >= nb) {
          in -= nb;
          ++g;
        }
        st->b = b;
        st->seq = s;
        st->tile = lo;
        st->g = g;
        st->j = in;
        break;
      }
      at += u;
    }
  }
}

// The producer warp: walks the span's segments, publishes each, copies its query rows (one copy a
// token; a tile of more than RowTok tokens fills both buffers, else they alternate) and its blocks'
// K and V regions, Sm::kStages ahead; the span's record for the join at the end.
template <typename Sm, typename Bar, int RowTok, typename Wait>
__device__ __forceinline__ void produce(const DenseParams& p, uint8_t* smem, const Bar& bars, const Start& start, Seg* segs,
                                        const CUtensorMap& kv_map, const CUtensorMap& q_map, Wait wwait) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) {
    prefetch_tensormap(&kv_map);
    prefetch_tensormap(&q_map);
  }
  const uint64_t qpol = policy_evict_first();
  int64_t left = start.count, at = start.first;
  const int64_t total = start.total, spans = total < kSpans ? total : kSpans;
  int b = start.b, tile = start.tile, g = start.g, j = start.j;
  int4 rec = make_int4(0, 0, 0, 0);
  int blocks = 0, k = 0;
  uint32_t qn = 0, qused = 0;  // bit x: parity of the copies into query buffer x; whether there was one
  bool ok = true, bad;
  Seq s{};
  if (left > 0) s = start.seq;
  for (; left > 0 && ok; ++k) {
    while (s.ql == 0) s = load_seq(p, ++b, &bad);  // units are left: a sequence with some follows
    const int i0 = tile << p.tile_log2, ntok = min(p.tile_tok, s.ql - i0);
    const int p0 = s.L - s.ql + i0, nb = (p0 + ntok - 1) / kBS + 1;
    const int n = static_cast<int>(nb - j < left ? nb - j : left);
    const int32_t* row = p.block_table + static_cast<int64_t>(b) * p.maxb;
    int next = lane < n ? row[j + lane] : 0;  // page ids, 32 at a time, loaded one round ahead
    const int ms = k % kSegs;
    if (!(ok = wwait(&bars.seg_empty[ms], (static_cast<uint32_t>(k / kSegs) & 1u) ^ 1u))) break;
    Seg& m = segs[ms];
    if (lane == 0) {
      m.n = n;
      m.j0 = j;
      m.t0 = s.q0 + i0;
      m.ntok = ntok;
      m.p0 = p0;
      m.g = g;
      m.part = j == 0 && n == nb ? -1 : (j == 0 ? 1 : 0);
      m.bad = 0x7fffffff;
      m.cut = p0 + ntok - j * kBS;
      mbar_arrive(&bars.seg_full[ms]);
    }
    // the query rows: one copy a token; a tile of more than 8 tokens fills both buffers
    const int x0 = ntok > RowTok ? 0 : k & 1, nx = ntok > RowTok ? 2 : 1;
    for (int x = x0; x < x0 + nx && ok; ++x) {
      const int tk = nx == 2 ? (x == 0 ? RowTok : ntok - RowTok) : ntok;
      if (!(ok = wwait(&bars.q_empty[x], ((qn >> x) & 1u) ^ 1u))) break;
      qn ^= 1u << x;
      qused |= 1u << x;
      if (lane == 0) mbar_arrive_expect_tx(&bars.q_full[x], static_cast<uint32_t>(tk) * kHPG * kD);
      __syncwarp();
      if (lane < tk)
        tma_load_2d(smem + Sm::kOffQ + static_cast<size_t>(x) * Sm::kQTile + lane * kHPG * kD, &q_map, 0,
                    (s.q0 + i0 + (nx == 2 ? RowTok * x : 0) + lane) * kQHeads + g * kHPG, &bars.q_full[x], qpol);
    }
    for (int i = 0; i < n && ok; i += 32) {
      const int pages = next, c = min(32, n - i);
      if (i + 32 + lane < n) next = row[j + i + 32 + lane];
      const uint32_t bads = __ballot_sync(0xffffffffu, lane < c && (pages < 0 || pages >= p.num_pages));
      if (bads != 0 && lane == 0) {
        set_status(p.status, MSA_ERR_DEVICE_FAULT);
        const int pos = (j + i + __ffs(bads) - 1) * kBS;
        if (pos < m.bad) {  // before the block's copy: its users see it
          m.bad = pos;
          m.cut = min(m.cut, pos - j * kBS);
        }
      }
      for (int u = 0; u < c; ++u, ++blocks) {
        const int st = blocks % Sm::kStages;
        int ph = __shfl_sync(0xffffffffu, pages, u);
        if (ph < 0 || ph >= p.num_pages) ph = 0;  // any page: the rows that see it are zeroed, its V taken as zeros
        if (!(ok = wwait(&bars.raw_empty[st], (static_cast<uint32_t>(blocks / Sm::kStages) & 1u) ^ 1u))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars.raw_full[st], kStageBytes);
          tma_load_3d(smem + Sm::kOffStage + static_cast<size_t>(st) * kStageBytes, &kv_map, 0, 2 * g * (kRegion / kD),
                      ph, &bars.raw_full[st]);
        }
        __syncwarp();
      }
    }
    if (j == 0 && n < nb) {  // starts here, ends in a later span: the one that holds its last unit
      const int64_t end = at + nb;
      rec = make_int4(static_cast<int>((end * spans - 1) / total) - static_cast<int>(blockIdx.x) + 1, s.q0 + i0, ntok, g);
    }
    left -= n;
    at += n;
    j = 0;
    if (++g == kGroups) {
      g = 0;
      if ((++tile << p.tile_log2) >= s.ql) {
        tile = 0;
        s.ql = 0;
      }
    }
  }
  if (lane == 0) p.rec[blockIdx.x] = rec;
  if (ok && wwait(&bars.seg_empty[k % kSegs], (static_cast<uint32_t>(k / kSegs) & 1u) ^ 1u) && lane == 0) {
    segs[k % kSegs].n = -1;
    mbar_arrive(&bars.seg_full[k % kSegs]);
  }
  // never leave while a copy into this CTA's shared memory may still be in flight
  if (lane == 0) {
    for (int i = blocks > Sm::kStages ? blocks - Sm::kStages : 0; i < blocks; ++i)
      if (!mbar_wait_bounded(&bars.raw_full[i % Sm::kStages], static_cast<uint32_t>(i / Sm::kStages) & 1u, kWaitLimitNs, nullptr))
        set_status(p.status, MSA_ERR_TIMEOUT);
    for (int x = 0; x < 2; ++x)
      if ((qused >> x & 1u) != 0 && !mbar_wait_bounded(&bars.q_full[x], ((qn >> x) & 1u) ^ 1u, kWaitLimitNs, nullptr))
        set_status(p.status, MSA_ERR_TIMEOUT);
  }
}

// ------------------------------------------------------------------ rows in, tiles out -
// The integer pipe is the busiest one of these kernels (the dequant's permutes), so the rows and tiles
// are addressed by shared-memory addresses with one exclusive-or a 16-byte chunk (a swizzled row's
// chunks are those of its first one xor-ed with the chunk's number), and a scale's table entry
// (byte x 8 + table) by one dot product instead of a shift, a mask and an add.
__device__ __forceinline__ uint4 lds128_at(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64_at(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128_at(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Where key row r's first code chunk and its scales stand in a staged (128-byte swizzled) region.
struct RowAt {
  uint32_t codes, scales;
  __device__ __forceinline__ RowAt(uint32_t region, int r)
      : codes(region + sw128_phys(static_cast<uint32_t>(r * kRowCodes))),
        scales(region + sw128_phys(static_cast<uint32_t>(kScaleOff + r * kRowScales))) {}
};
__device__ __forceinline__ void load_row_at(const RowAt& at, uint32_t stage, RawRow& raw) {
  raw.sc = lds64_at(at.scales + stage);
  const uint32_t a = at.codes + stage;
#pragma unroll
  for (int q = 0; q < 4; ++q) raw.c[q] = lds128_at(a ^ (q << 4));
}

__device__ __forceinline__ uint2 lut_entry(uint32_t scales, int k, uint32_t lut) {
  uint2 e;
  asm("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(e.x), "=r"(e.y) : "r"(__dp4a(scales, 8u << (8 * k), lut)));
  return e;
}
__device__ __forceinline__ void dequant_quarter(const RawRow& raw, int q, uint32_t lut, uint32_t (&w)[8]) {
  const uint32_t s = q < 2 ? raw.sc.x : raw.sc.y;
  const uint2 e0 = lut_entry(s, 2 * (q & 1), lut), e1 = lut_entry(s, 2 * (q & 1) + 1, lut);
  dq8(raw.c[q].x, e0, w[0], w[1]);
  dq8(raw.c[q].y, e0, w[2], w[3]);
  dq8(raw.c[q].z, e1, w[4], w[5]);
  dq8(raw.c[q].w, e1, w[6], w[7]);
}

// Persistent, one CTA a span. Warp roles:
//  producer — walks the span's segments (a segment: the part of one (tile, group) inside the span),
//             publishes each in a ring, copies its query rows and its blocks' K and V regions;
//  dequant  — two warpgroups that take blocks in turn, thread = key: the block's K rows to an E4M3 K-major
//             tile, then its V rows to an f16 tile read with the dims contiguous; rows after the tile's
//             last position become zeros in V (with K and V on a warpgroup each, V's set the pace: 32 x 16K
//             of 8 tokens 115.8 us instead of 111.3);
//  S issuer — S = Q K^T (E4M3, M 128 rows x N 128 keys) into one of two score slots in TMEM;
//  softmax  — two warpgroups, one per slot, thread = row: P in f16 over the scores' own columns;
//  PV issuer— O[slot] += P V (f16, A = P in TMEM, N 128 dims).
// A block is two steps of 64 keys: a half's scores can be overwritten as soon as its own PV is done, so
// that the next block's first half is scored while the softmax works on this one's second (with whole
// blocks each slot's chain S, softmax, PV, S left the softmax waiting 40 % of the time).
// A tile of more than 8 tokens is two row tiles: slot = row tile, every block goes through both, and
// its K and V are dequantised once for both. A tile of at most 8 tokens alternates its blocks over
// the slots; the two slots' sums are joined when the segment ends. Either way the softmax of one
// slot runs while the tensor core works on the other. Every wait is bounded (MSA_ERR_TIMEOUT, then
// every role leaves); nothing traps.
// The roles' order in the source is measured: the hot loops together fill the instruction cache, and
// other orders of the same code took up to 670 us where this one takes 563 for a 2,048-token prompt.
// 20 warps leave 96 registers a thread, and k_dense<false> spills 12 bytes, k_dense<true> 16.
template <bool kTwo>
__global__ void __launch_bounds__(kThreads, 1)
    k_dense(const DenseParams p, const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap q_map) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const Bars bars(smem);
  Seg* segs = reinterpret_cast<Seg*>(smem + Smem::kOffSeg);
  Start* start = reinterpret_cast<Start*>(smem + Smem::kOffStart);
  uint2* lut = reinterpret_cast<uint2*>(smem + Smem::kOffLut);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Smem::kOffMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Smem::kOffMisc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&bars.seg_full[i], 1);
      mbar_init(&bars.seg_empty[i], kSegUsers);
    }
    for (int i = 0; i < Smem::kStages; ++i) {
      mbar_init(&bars.raw_full[i], 1);
      mbar_init(&bars.raw_empty[i], 4);  // the block's dequant warpgroup
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.q_full[i], 1);
      mbar_init(&bars.q_empty[i], 1);
      mbar_init(&bars.k_full[i], 4);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.v_full[i], 4);
      mbar_init(&bars.v_empty[i], 1);
      mbar_init(&bars.fin[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_full[i], 4);
      mbar_init(&bars.pv_done[i], 1);
    }
    mbar_init(bars.o_free, 8);
    mbar_init(bars.ml, 8);
    fence_mbar_init();
    *abort_flag = 0;
  }
  {
    // the query tiles start as zeros: rows of absent tokens then hold finite values
    uint4* qz = reinterpret_cast<uint4*>(smem + Smem::kOffQ);
    for (int i = tid; i < 2 * Smem::kQTile / 16; i += kThreads) qz[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (warp == 3) tmem_alloc(tmem_slot, kTmemCols);
  build_dequant_lut(lut, tid, kThreads);
  fence_proxy_async_smem();
  grid_dependency_wait();  // what ran before may have written the batch, the cache or the queries
  find_start(p, start, reinterpret_cast<int64_t*>(smem + Smem::kOffScan), kThreads);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_launch_dependents();  // the join's CTAs take the SMs' places as this grid's leave (beside one there is no room)

  auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {  // a warp's bounded wait
    if (warp_wait(bar, parity, abort_flag)) return true;
    if (lane == 0) {
      if (!*abort_flag) set_status(p.status, MSA_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    return false;
  };

  if (warp < kWarpDq) {
    if (warp == kWarpProd) {
      produce<Smem, Bars, kTileTok>(p, smem, bars, *start, segs, kv_map, q_map, wwait);
    } else if (warp == kWarpS) {
      // ---- S = Q K^T, an elected lane ------------------------------------------------------------------
      constexpr uint32_t idesc = idesc_e4m3_f32(kRows, kHalf);
      const uint64_t dq0 = sw128_kmajor_desc(smem_u32(smem + Smem::kOffQ)), dk0 = sw128_kmajor_desc(smem_u32(smem + Smem::kOffK));
      uint32_t par0 = 0, par1 = 0, qn = 0;  // parities of the slots' blocks; bit x: of query buffer x's tiles
      int blocks = 0;
      constexpr uint32_t kQStep = Smem::kQTile >> 4;
      // the scores of half h of the block into slot x (both known to the compiler: an issuer's own
      // instructions are on every step's path)
      auto step = [&](auto xc, auto hc, uint64_t dk, uint64_t dq, int kb, bool last) -> bool {
        constexpr int x = decltype(xc)::value, hx = decltype(hc)::value;
        uint32_t& par = x == 0 ? par0 : par1;
        if (!wwait(&bars.pv_done[2 * x + hx], par ^ 1u)) return false;  // the half's P has been read
        if (hx == 1) par ^= 1u;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // K = 32 dims per MMA: +32 B in both operands' atoms
            tc_mma_f8(tmem + 128u * x + kHalf * hx, dq + 2 * kk, dk + static_cast<uint32_t>(hx * kHalf * kD >> 4) + 2 * kk,
                      idesc, kk > 0 ? 1u : 0u);
          tc_commit(&bars.s_full[2 * x + hx]);
          if (last) tc_commit(&bars.k_empty[kb]);
        }
        __syncwarp();
        return true;
      };
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const int ms = k % kSegs;
        if (!wwait(&bars.seg_full[ms], static_cast<uint32_t>(k / kSegs) & 1u)) break;
        const int n = segs[ms].n;
        if (n < 0) break;
        const bool two = kTwo && segs[ms].ntok > kTileTok;
        for (int x = 0; x < 2; ++x)
          if (two || x == (k & 1)) {
            ok = ok && wwait(&bars.q_full[x], (qn >> x) & 1u);
            qn ^= 1u << x;
          }
        for (int i = 0; i < n && ok; ++i, ++blocks) {
          const int kb = blocks & 1;
          if (!(ok = wwait(&bars.k_full[kb], static_cast<uint32_t>(blocks >> 1) & 1u))) break;
          const uint64_t dk = dk0 + static_cast<uint32_t>(kb * kKTile >> 4), dqk = dq0 + (k & 1) * kQStep;
          if (two)
            ok = step(kX0, kX0, dk, dq0, kb, false) && step(kX1, kX0, dk, dq0 + kQStep, kb, false) &&
                 step(kX0, kX1, dk, dq0, kb, false) && step(kX1, kX1, dk, dq0 + kQStep, kb, true);
          else if ((i & 1) == 0)
            ok = step(kX0, kX0, dk, dqk, kb, false) && step(kX0, kX1, dk, dqk, kb, true);
          else
            ok = step(kX1, kX0, dk, dqk, kb, false) && step(kX1, kX1, dk, dqk, kb, true);
        }
        for (int x = 0; x < 2; ++x)
          if ((two || x == (k & 1)) && elect_one()) tc_commit(&bars.q_empty[x]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.seg_empty[ms]);
      }
      // nothing of this thread's is in flight when the CTA ends
      if (elect_one()) tc_commit(&bars.fin[0]);
      __syncwarp();
      if (!mbar_wait_bounded(&bars.fin[0], 0u, kWaitLimitNs, nullptr)) set_status(p.status, MSA_ERR_TIMEOUT);
    } else if (warp == kWarpPv) {
      // ---- O += P V, an elected lane -------------------------------------------------------------------
      constexpr uint32_t idesc = idesc_f16_f32_bmn(kRows, kD);
      const uint64_t dv0 = sw128_mnmajor_desc(smem_u32(smem + Smem::kOffV), kVLbo, kVSbo);
      uint32_t par0 = 0, par1 = 0;
      int blocks = 0;
      auto step = [&](auto xc, auto hc, uint64_t dv, bool first, int vb, bool last) -> bool {
        constexpr int x = decltype(xc)::value, hx = decltype(hc)::value;
        uint32_t& par = x == 0 ? par0 : par1;
        if (!wwait(&bars.p_full[2 * x + hx], par)) return false;
        if (hx == 1) par ^= 1u;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // K = 16 keys per MMA: 8 columns of P, two 8-key groups of V
            tc_mma_f16_ta(tmem + kColO + 128u * x, tmem + 128u * x + kHalf * hx + 8 * kk,
                          dv + ((2 * kVSbo) >> 4) * (4 * hx + kk), idesc, (!first || kk > 0) ? 1u : 0u);
          tc_commit(&bars.pv_done[2 * x + hx]);
          if (last) tc_commit(&bars.v_empty[vb]);
        }
        __syncwarp();
        return true;
      };
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const int ms = k % kSegs;
        if (!wwait(&bars.seg_full[ms], static_cast<uint32_t>(k / kSegs) & 1u)) break;
        const int n = segs[ms].n;
        if (n < 0) break;
        const bool two = kTwo && segs[ms].ntok > kTileTok;
        if (!wwait(bars.o_free, (static_cast<uint32_t>(k) & 1u) ^ 1u)) break;  // the last segment's O has been read
        for (int i = 0; i < n && ok; ++i, ++blocks) {
          const int vb = blocks & 1;
          if (!(ok = wwait(&bars.v_full[vb], static_cast<uint32_t>(blocks >> 1) & 1u))) break;
          const uint64_t dv = dv0 + static_cast<uint32_t>(vb * kVTile >> 4);
          const bool first = two ? i == 0 : i < 2;
          if (two)
            ok = step(kX0, kX0, dv, first, vb, false) && step(kX1, kX0, dv, first, vb, false) &&
                 step(kX0, kX1, dv, false, vb, false) && step(kX1, kX1, dv, false, vb, true);
          else if ((i & 1) == 0)
            ok = step(kX0, kX0, dv, first, vb, false) && step(kX0, kX1, dv, false, vb, true);
          else
            ok = step(kX1, kX0, dv, first, vb, false) && step(kX1, kX1, dv, false, vb, true);
        }
        if (lane == 0) mbar_arrive(&bars.seg_empty[ms]);
      }
      if (elect_one()) tc_commit(&bars.fin[1]);
      __syncwarp();
      if (!mbar_wait_bounded(&bars.fin[1], 0u, kWaitLimitNs, nullptr)) set_status(p.status, MSA_ERR_TIMEOUT);
    }
  } else if (warp < kWarpSm) {
    // ---- dequant warpgroup w: blocks g with g % 2 == w, thread = key row ---------------------------
    const int w = (warp - kWarpDq) >> 2, r = tid & 127;
    const uint32_t lut32 = smem_u32(lut);
    const RowAt at_k(smem_u32(smem + Smem::kOffStage), r), at_v(smem_u32(smem + Smem::kOffStage) + kRegion, r);
    // chunk 0 of row r of tile w, in the swizzle's place
    const uint32_t kt = smem_u32(smem + Smem::kOffK) + w * kKTile + sw128_chunk_off(r, 0);
    const uint32_t vt = smem_u32(smem + Smem::kOffV) + w * kVTile + (r >> 3) * kVSbo + (r & 7) * 128 + ((r & 7) << 4);
    int first = 0, st = w;  // the segment's first block; this block's stage
    uint32_t raw_par = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int ms = k % kSegs;
      if (!wwait(&bars.seg_full[ms], static_cast<uint32_t>(k / kSegs) & 1u)) break;
      const int n = segs[ms].n;
      if (n < 0) break;
      for (int g = first + ((w ^ first) & 1); g < first + n; g += 2) {
        const uint32_t free = (static_cast<uint32_t>(g >> 1) & 1u) ^ 1u;
        if (!(ok = wwait(&bars.raw_full[st], raw_par))) break;
        RawRow raw;
        load_row_at(at_k, st * kStageBytes, raw);
        if (!(ok = wwait(&bars.k_empty[w], free))) break;
#pragma unroll
        for (int qd = 0; qd < 4; ++qd) {
          uint32_t u[8];
          dequant_quarter(raw, qd, lut32, u);
          sts128_at(kt ^ ((2 * qd) << 4), u[0], u[1], u[2], u[3]);
          sts128_at(kt ^ ((2 * qd + 1) << 4), u[4], u[5], u[6], u[7]);
        }
        fence_proxy_async_smem();  // the tiles are read by the tensor core
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.k_full[w]);
        load_row_at(at_v, st * kStageBytes, raw);
        // after the last position, or for a bad page id, anything may stand there: 0 x NaN is NaN
        if ((g - first) * kBS + r >= segs[ms].cut) {
          raw.c[0] = raw.c[1] = raw.c[2] = raw.c[3] = make_uint4(0u, 0u, 0u, 0u);
          raw.sc = make_uint2(0u, 0u);
        }
        if (!(ok = wwait(&bars.v_empty[w], free))) break;
#pragma unroll
        for (int qd = 0; qd < 4; ++qd) {
          uint32_t u[8];
          dequant_quarter(raw, qd, lut32, u);
#pragma unroll
          for (int hh = 0; hh < 4; ++hh) {  // dims 32 qd + 8 hh .. + 7 = 16-byte chunk cc of the row
            const int cc = 4 * qd + hh;
            sts128_at((vt ^ ((cc & 7) << 4)) + (cc >> 3) * kVLbo, cvt_f16x2_e4m3x2(u[2 * hh]),
                      cvt_f16x2_e4m3x2(u[2 * hh] >> 16), cvt_f16x2_e4m3x2(u[2 * hh + 1]),
                      cvt_f16x2_e4m3x2(u[2 * hh + 1] >> 16));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          // only now: a stage released right after the rows' loads could be refilled before they had
          // executed (nothing used them before the wait on the tile)
          mbar_arrive(&bars.raw_empty[st]);
          mbar_arrive(&bars.v_full[w]);
        }
        st += 2;
        if (st >= Smem::kStages) {
          st -= Smem::kStages;
          raw_par ^= 1u;
        }
      }
      first += n;
      if (ok && lane == 0) mbar_arrive(&bars.seg_empty[ms]);
    }
  } else {
    // ---- softmax warpgroup x (score slot x): thread = row 32 q + lane ---------------------------
    const int x = (warp - kWarpSm) >> 2, q = warp & 3;
    const int row = 32 * q + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
    const uint32_t ts = tmem + lanes + 128u * static_cast<uint32_t>(x);
    const float c = p.scale_log2;
    float2* mls = reinterpret_cast<float2*>(smem + Smem::kOffMl);
    uint32_t steps = 0;  // bit y: parity of slot y's blocks
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int ms = k % kSegs;
      if (!wwait(&bars.seg_full[ms], static_cast<uint32_t>(k / kSegs) & 1u)) break;
      const Seg& m = segs[ms];
      const int n = m.n;
      if (n < 0) break;
      const bool two = kTwo && m.ntok > kTileTok;
      const int tok = (row >> 4) + (two ? kTileTok * x : 0);  // this row's token in the tile
      const bool real = tok < m.ntok;
      const int ptok = m.p0 + min(tok, m.ntok - 1);           // absent rows run along with the last token
      const bool idle = !__any_sync(0xffffffffu, real);       // no row of this warp is there
      float ref = -CUDART_INF_F, l = 0.f;
      const int stride = two ? 1 : 2;
      const int mysteps = two ? n : (n - x + 1) >> 1;
      for (int i = two ? 0 : x, z = 0; z < mysteps; i += stride, ++z) {
        const int rel = ptok - (m.j0 + i) * kBS;                // keys after rel are masked
        const bool full = __all_sync(0xffffffffu, rel >= kBS - 1);
        const uint32_t par = ((steps >> x) + z) & 1u;
#pragma unroll 1
        for (int hx = 0; hx < 2; ++hx) {
          if (!(ok = wwait(&bars.s_full[2 * x + hx], par))) break;
          tc_fence_after();
          if (!idle) {
            const uint32_t th = ts + kHalf * hx;
            // P = 2^(s c - ref) over the scores' own columns, in one load and one store of the half (each waits
            // its turn behind the tensor core's accesses: with 16 keys at a time a prompt took 861 us instead of
            // 570). P and its sum are fp32 (the f16x2 exp2 is off by up to 2^-11, which the log-sum-exp of a few
            // keys would show); P is rounded to f16 for the MMA alone. No maximum is taken while the half's sum
            // stays within kMostSum: every P is then inside f16, and the reference can stay.
            uint32_t r[kHalf], w[kHalf / 2];
            auto scores = [&]() {
              tmem_ld64(th, r);
              tmem_wait_ld();
              if (!full) {
#pragma unroll
                for (int u = 0; u < kHalf; ++u) r[u] = kHalf * hx + u > rel ? __float_as_uint(-CUDART_INF_F) : r[u];
              }
            };
            float s0, s1;
            auto powers = [&]() {
              const float mu = ref == -CUDART_INF_F ? 0.f : ref;
              s0 = s1 = 0.f;
#pragma unroll
              for (int u = 0; u < kHalf / 2; ++u) {
                float x0, x1;
                fma_f32x2(__uint_as_float(r[2 * u]), __uint_as_float(r[2 * u + 1]), c, c, -mu, -mu, x0, x1);
                x0 = fast_exp2(x0);
                x1 = fast_exp2(x1);
                add_f32x2(s0, s1, x0, x1);
                w[u] = pack_f16x2(x0, x1);
              }
            };
            // The segment's first half sets the reference. (With more code in the way, k_dense<true> is slower:
            // its first half takes the common path, twice.)
            const bool first = z == 0 && hx == 0;
            bool need = true;
            if (kTwo || !first) {
              scores();
              powers();
              need = !(s0 + s1 <= kMostSum) || ref == -CUDART_INF_F;
            }
            if (!kTwo && first || __any_sync(0xffffffffu, need)) {
              // ---- the reference moves to the half's maximum: what the row has so far shrinks by cf
              scores();
              float mx = -CUDART_INF_F;
#pragma unroll
              for (int u = 0; u < kHalf; u += 2) mx = max3f(mx, __uint_as_float(r[u]), __uint_as_float(r[u + 1]));
              mx = fmaf(mx, c, -kRaise);  // c > 0
              const float to = need && mx > ref ? mx : ref;
              const float cf = to == ref ? 1.f : fast_exp2(ref - to);
              ref = to;
              l *= cf;
              if (!first) {  // O, once the PV of this slot's last half has landed
                if (!(ok = wwait(&bars.pv_done[2 * x + (hx ^ 1)], hx == 0 ? par ^ 1u : par))) break;
                tc_fence_after();
#pragma unroll 1
                for (int d = 0; d < kD; d += 32) {
                  uint32_t o[32];
                  tmem_ld32(tmem + lanes + kColO + 128u * static_cast<uint32_t>(x) + d, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * cf);
                  tmem_st32(tmem + lanes + kColO + 128u * static_cast<uint32_t>(x) + d, o);
                }
              }
              scores();  // again, rather than kept across the sums of O
              powers();
            }
            l += s0 + s1;
            tmem_st32(th, w);
            if (!ok) break;
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.p_full[2 * x + hx]);
        }
        if (!ok) break;
      }
      if (!ok) break;
      const bool both = two || n > 1;  // slot 1 has blocks, too
      steps ^= two ? (n & 1 ? 3u : 0u) : (((n + 1) >> 1) & 1u) | (((n >> 1) & 1u) << 1);
      // ---- the segment's result: rows joined over the slots (a tile of at most 8 tokens) -----------
      float2* ml = mls + (k & 1) * 2 * kRows;
      ml[x * kRows + row] = make_float2(ref, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(bars.ml);
      if (!(ok = wwait(bars.ml, static_cast<uint32_t>(k) & 1u))) break;
#pragma unroll
      for (int y = 0; y < 2; ++y)  // the slots' last PVs
        if (two ? y == x : y == 0 || both) ok = ok && wwait(&bars.pv_done[2 * y + 1], ((steps >> y) & 1u) ^ 1u);
      if (!ok) break;
      tc_fence_after();
      float w0 = 1.f, w1 = 0.f;
      if (!two) {
        const float2 a = ml[row], d = ml[kRows + row];
        const float M = fmaxf(a.x, d.x);
        w0 = a.x == -CUDART_INF_F ? 0.f : fast_exp2(a.x - M);
        w1 = d.x == -CUDART_INF_F ? 0.f : fast_exp2(d.x - M);
        ref = M;
        l = w0 * a.y + w1 * d.y;
      }
      const bool bad = m.bad <= ptok;
      const float inv = m.part < 0 ? (bad || !(l > 0.f) && l == l ? 0.f : 1.f / l) : 1.f;
      const int64_t prow = m.part < 0 ? 0 : (static_cast<int64_t>(blockIdx.x) * 2 + m.part) * (p.tile_tok * kHPG) + tok * kHPG + (row & 15);
      const int64_t orow = static_cast<int64_t>(m.t0 + tok) * kQHeads + m.g * kHPG + (row & 15);
      // two slots: this warpgroup takes half the columns of both; else all columns of its own
      if (!idle) {
#pragma unroll 1
        for (int cc = two ? 0 : 2 * x; cc < (two ? 4 : 2 * x + 2); ++cc) {
          uint32_t o[32];
          if (two) {
            tmem_ld32(tmem + lanes + kColO + 128u * static_cast<uint32_t>(x) + 32 * cc, o);
            tmem_wait_ld();
          } else {
            tmem_ld32(tmem + lanes + kColO + 32 * cc, o);  // slot 0 has the segment's first block
            tmem_wait_ld();
#pragma unroll
            for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * w0);
            if (both) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t o1[16];
                tmem_ld16(tmem + lanes + kColO + 128 + 32 * cc + 16 * h, o1);
                tmem_wait_ld();
#pragma unroll
                for (int u = 0; u < 16; ++u)
                  o[16 * h + u] = __float_as_uint(fmaf(w1, __uint_as_float(o1[u]), __uint_as_float(o[16 * h + u])));
              }
            }
          }
          if (real) {
            if (m.part < 0) {
              uint4* dst = reinterpret_cast<uint4*>(p.out + orow * kD + 32 * cc);
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float v0 = __uint_as_float(o[8 * u + 2 * e]) * inv, v1 = __uint_as_float(o[8 * u + 2 * e + 1]) * inv;
                  w[e] = bad ? 0u : pack_bf16x2(v0, v1);
                }
                dst[u] = make_uint4(w[0], w[1], w[2], w[3]);
              }
            } else {
              uint4* dst = reinterpret_cast<uint4*>(p.part_o + prow * kD + 32 * cc);
#pragma unroll
              for (int u = 0; u < 8; ++u) dst[u] = make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
            }
          }
        }
      }
      if (real && (two || x == 0)) {
        if (m.part >= 0) {
          p.part_ml[prow] = make_float2(bad ? CUDART_NAN_F : ref, l);
        } else if (p.lse != nullptr) {
          p.lse[orow] = bad ? -CUDART_INF_F : (ref + __log2f(l)) * 0.69314718055994531f;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bars.o_free);
        mbar_arrive(&bars.seg_empty[ms]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------ one token a tile ----
// The same work for batches of at most one query token a sequence (16 rows a tile), transposed: the
// block's 128 keys are the MMAs' M and the query rows their N, so that the tensor core, the softmax and
// shared memory see only the rows there are.
//  S^T = K Q^T: A = the K rows, E4M3, put into TMEM by the dequant warps; B = the query rows.
//  O^T += V^T P^T: A = the V rows, E4M3, read with the dims along M; B = P^T as three E5M2 parts in rows
//  0 .. 15, 16 .. 31 and 32 .. 47: P is rounded to f16, its upper byte is the first part (two bits after
//  the leading one, what is left below 2^-2 of that), the upper byte of what is left the second (below
//  2^-5), what is left then, times 32 and rounded to nearest, the third: off by 2^-9 of P at most, and by
//  no more than 2^-22 where P is small (E5M2's subnormals are 2^-16 apart). The reference is a running
//  maximum less 10 (log2), moved when a score passes it by 15: the largest P lies between 2^10 and 2^15, so
//  that 2^-22 is 2^-32 of it and keys far below one that they outweigh together keep their weight; a maximum
//  may grow by 2^5 before the sums are rescaled. (Two E4M3 parts, off by 2^-17 of the largest P, lost
//  the keys 17 bits below a heavy first one, and saved 4 us of a 32 x 32K call. With room for a growth of 2^2 a third of the blocks
//  of scores of standard deviation 2 rescaled, and cost 10 us of a 32 x 32K call.)
// Two dequant warpgroups take blocks in turn (K rows, then V rows), and two softmax warpgroups, each with
// its own reference, sum and O^T; these are joined at a segment's end. What bounds it: a 32 x 32K call
// takes 132 us where its bytes take 89. No unit is full: the integer pipe is 53 % busy (the dequant's permutes: 7
// instructions for 8 elements), the issue slots 56 %, DRAM 69 %; the dequant warps, two a scheduler, wait for
// their table look-ups. More warps (three warpgroups of either kind, or K and V apart) were slower, by 20 %
// and more.
namespace few {

constexpr int kWarpProd = 0, kWarpS = 1, kWarpPv = 2, kWarpTmem = 3, kWarpDq = 4, kWarpSm = 12;
constexpr int kWarps = 20, kThreads = 32 * kWarps;
constexpr int kSegUsers = 1 + 1 + 8 + 8;
constexpr int kParts = 3;                   // of a P
constexpr float kUp = 10.0f;                // P = 2^(z - max + kUp)
constexpr float kRescaleLog2 = 15.0f;       // the largest exponent of a P: 2^15 < 57,344, the E5M2 maximum
constexpr float kLastScale = 32.0f;         // of the last part: below 2^10 unscaled (P < 2^16)
constexpr uint32_t kLastScale2 = 0x50005000u; // f16x2 {32, 32}
constexpr int kBarVote = 1, kBarX = 3;      // named barriers of softmax warpgroup x: kBarVote + x, kBarX + x

struct Sm {
  static constexpr int kN = kHPG;              // query rows
  static constexpr int kStages = 6;            // even: a dequant warpgroup steps by two
  static constexpr int kQTile = kN * kD;
  static constexpr int kPTile = kParts * kN * kBS;  // the parts' rows of 128 keys
  static constexpr int kVTile = kBS * kD;      // E4M3
  static constexpr size_t kOffStage = 0;
  static constexpr size_t kOffV = kOffStage + kStages * static_cast<size_t>(kStageBytes);  // [4] V tiles
  static constexpr size_t kOffQ = kOffV + 4 * static_cast<size_t>(kVTile);
  static constexpr size_t kOffP = kOffQ + 2 * static_cast<size_t>(kQTile);                 // [4] P^T tiles
  static constexpr size_t kOffLut = kOffP + 4 * static_cast<size_t>(kPTile);
  static constexpr size_t kOffMax = kOffLut + 256 * 8;            // [2 wg][4 warps][kN] block maxima of a rescale
  static constexpr size_t kOffCf = kOffMax + 2 * 4 * kN * 4;      // [2 wg][kN] its factors
  static constexpr size_t kOffL = kOffCf + 2 * kN * 4;            // [2 parities][2 wg][4 warps][kN] sums
  static constexpr size_t kOffRef = kOffL + 2 * 2 * 4 * kN * 4;   // [2 parities][2 wg][kN] references
  static constexpr size_t kOffSeg = kOffRef + 2 * 2 * kN * 4;
  static constexpr size_t kOffStart = kOffSeg + kSegs * sizeof(Seg);
  static constexpr size_t kOffScan = kOffStart + sizeof(Start);
  static constexpr size_t kOffBar = kOffScan + kWarps * 8;
  static constexpr int kNumBars = 2 * kSegs + 2 * kStages + 4 + 2 + 2 + 4 + 4 + 2 + 2;
  static constexpr size_t kOffMisc = kOffBar + 8 * kNumBars;
  static constexpr size_t kBytes = 1024 + kOffMisc + 16;
  // TMEM columns: K tiles [2] (32 each), S^T [2] (kN each), O^T [2] (64 each, kParts kN in use)
  static constexpr uint32_t kColS = 64, kColO = 128, kOStep = 64;
  static constexpr uint32_t kTmemCols = 256;
  static_assert(kOffV % 1024 == 0 && kOffQ % 1024 == 0 && kOffP % 1024 == 0 && kQTile % 1024 == 0 && kPTile % 1024 == 0,
                "swizzled tiles start on 1024-B boundaries");
  static_assert(kOffStart % 8 == 0 && kOffBar % 8 == 0 && kBytes <= 232448, "shared memory per CTA");
  static_assert(kColS + 2 * kN <= kColO && kParts * kN <= kOStep && kColO + 2 * kOStep <= kTmemCols, "TMEM columns");
};

// Block g of the span (counted over its segments) uses K tile, score slot and O^T g % 2, V and P^T
// tiles g % 4. One barrier stands for all that an MMA needs, one commit for all that it frees, so
// that an issuer's block is a wait, four MMAs and a commit (with a barrier each, two waits and two
// or three commits, the issuers' own ~1,000 cycles a block set the pace):
//  s_in[g % 2]   K(g) is in TMEM (4 dequant warps) and S^T(g - 2) has been read (4 softmax warps)
//  s_out[g % 2]  S^T(g) is there, and K(g)'s tile free
//  pv_in[g % 4]  V(g) (4 dequant warps) and P^T(g) (4 softmax warps) are there
//  pv_out[g % 4] O^T has block g, and V(g)'s and P^T(g)'s tiles are free
struct FewBars {
  uint64_t *seg_full, *seg_empty, *raw_full, *raw_empty, *q_full, *q_empty, *s_in, *s_out, *pv_in, *pv_out, *o_free, *ml,
      *fin;
  __device__ explicit FewBars(uint8_t* smem) {
    using S = Sm;
    uint64_t* b = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
    auto take = [&](int n) {
      uint64_t* r = b;
      b += n;
      return r;
    };
    seg_full = take(kSegs);
    seg_empty = take(kSegs);
    raw_full = take(S::kStages);
    raw_empty = take(S::kStages);
    q_full = take(2);
    q_empty = take(2);
    s_in = take(2);
    s_out = take(2);
    pv_in = take(4);
    pv_out = take(4);
    o_free = take(1);
    ml = take(1);
    fin = take(2);
  }
};

__global__ void __launch_bounds__(kThreads, 1)
    k_dense_few(const DenseParams p, const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap q_map) {
  using S = Sm;
  constexpr int kN = S::kN;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const FewBars bars(smem);
  Seg* segs = reinterpret_cast<Seg*>(smem + S::kOffSeg);
  Start* start = reinterpret_cast<Start*>(smem + S::kOffStart);
  uint2* lut = reinterpret_cast<uint2*>(smem + S::kOffLut);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kOffMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffMisc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&bars.seg_full[i], 1);
      mbar_init(&bars.seg_empty[i], kSegUsers);
    }
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&bars.raw_full[i], 1);
      mbar_init(&bars.raw_empty[i], 4);  // the block's dequant warpgroup
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.q_full[i], 1);
      mbar_init(&bars.q_empty[i], 1);
      mbar_init(&bars.s_in[i], 8);
      mbar_init(&bars.s_out[i], 1);
      mbar_init(&bars.fin[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars.pv_in[i], 8);
      mbar_init(&bars.pv_out[i], 1);
    }
    mbar_init(bars.o_free, 8);
    mbar_init(bars.ml, 8);
    fence_mbar_init();
    *abort_flag = 0;
  }
  if (warp == kWarpTmem) tmem_alloc(tmem_slot, S::kTmemCols);
  build_dequant_lut(lut, tid, kThreads);
  fence_proxy_async_smem();
  grid_dependency_wait();  // what ran before may have written the batch, the cache or the queries
  find_start(p, start, reinterpret_cast<int64_t*>(smem + S::kOffScan), kThreads);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_launch_dependents();  // the join's CTAs take the SMs' places as this grid's leave (beside one there is no room)

  auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {  // a warp's bounded wait
    if (warp_wait(bar, parity, abort_flag)) return true;
    if (lane == 0) {
      if (!*abort_flag) set_status(p.status, MSA_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    return false;
  };

  if (warp == kWarpProd) {
    produce<S, FewBars, 1>(p, smem, bars, *start, segs, kv_map, q_map, wwait);
  } else if (warp == kWarpS) {
    // ---- S^T = K Q^T, an elected lane ------------------------------------------------------------------
    constexpr uint32_t idesc = idesc_e4m3_f32(kBS, kN);
    int g = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int ms = k % kSegs;
      if (!wwait(&bars.seg_full[ms], static_cast<uint32_t>(k / kSegs) & 1u)) break;
      const int n = segs[ms].n;
      if (n < 0) break;
      const uint64_t dq = sw128_kmajor_desc(smem_u32(smem + S::kOffQ + static_cast<size_t>(k & 1) * S::kQTile));
      if (!wwait(&bars.q_full[k & 1], static_cast<uint32_t>(k >> 1) & 1u)) break;
      for (const int end = g + n; g < end; ++g) {
        const uint32_t x = g & 1;
        if (!(ok = wwait(&bars.s_in[x], static_cast<uint32_t>(g >> 1) & 1u))) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // K = 32 dims per MMA: 8 TMEM columns of A, +32 B of B
            tc_mma_f8_ta(tmem + S::kColS + kN * x, tmem + 32 * x + 8 * kk, dq + 2 * kk, idesc, kk > 0 ? 1u : 0u);
          tc_commit(&bars.s_out[x]);
        }
        __syncwarp();
      }
      if (elect_one()) tc_commit(&bars.q_empty[k & 1]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.seg_empty[ms]);
    }
    // nothing of this thread's is in flight when the CTA ends
    if (elect_one()) tc_commit(&bars.fin[0]);
    __syncwarp();
    if (!mbar_wait_bounded(&bars.fin[0], 0u, kWaitLimitNs, nullptr)) set_status(p.status, MSA_ERR_TIMEOUT);
  } else if (warp == kWarpPv) {
    // ---- O^T += V^T P^T, an elected lane ---------------------------------------------------------------
    constexpr uint32_t idesc = idesc_e4m3_e5m2_f32_amn(kD, kParts * kN);
    const uint64_t dv0 = sw128_mnmajor8_desc(smem_u32(smem + S::kOffV)), dp0 = sw128_kmajor_desc(smem_u32(smem + S::kOffP));
    int g = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int ms = k % kSegs;
      if (!wwait(&bars.seg_full[ms], static_cast<uint32_t>(k / kSegs) & 1u)) break;
      const int n = segs[ms].n;
      if (n < 0) break;
      if (!wwait(bars.o_free, (static_cast<uint32_t>(k) & 1u) ^ 1u)) break;  // the last segment's O^T has been read
      for (int i = 0; i < n; ++i, ++g) {
        const int y = g & 3;
        if (!(ok = wwait(&bars.pv_in[y], static_cast<uint32_t>(g >> 2) & 1u))) break;
        tc_fence_after();
        const uint64_t dv = dv0 + static_cast<uint32_t>(y * S::kVTile >> 4), dp = dp0 + static_cast<uint32_t>(y * S::kPTile >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // K = 32 keys per MMA: four 8-key groups of V (4 KB), +32 B of P^T
            tc_mma_f8(tmem + S::kColO + S::kOStep * (g & 1), dv + (4096 >> 4) * kk, dp + 2 * kk, idesc,
                      (i > 1 || kk > 0) ? 1u : 0u);
          tc_commit(&bars.pv_out[y]);
        }
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(&bars.seg_empty[ms]);
    }
    if (elect_one()) tc_commit(&bars.fin[1]);
    __syncwarp();
    if (!mbar_wait_bounded(&bars.fin[1], 0u, kWaitLimitNs, nullptr)) set_status(p.status, MSA_ERR_TIMEOUT);
  } else if (warp >= kWarpDq && warp < kWarpSm) {
    // ---- dequant warpgroup w: blocks g with g % 2 == w ---------------------------------------------
    const int w = (warp - kWarpDq) >> 2, q = warp & 3;
    const int key_k = 32 * q + kappa(lane);                          // K row -> TMEM lane 32 q + lane
    const int vpos = 32 * q + lane;                                  // V tile row: the key position
    const int key_v = 32 * q + kappa((lane >> 2) + 8 * (lane & 3));  // the key at that position
    const uint32_t tk = tmem + (static_cast<uint32_t>(32 * q) << 16) + 32 * w;
    const uint32_t lut32 = smem_u32(lut), stage0 = smem_u32(smem + S::kOffStage);
    const RowAt at_k(stage0, key_k), at_v(stage0 + kRegion, key_v);
    // chunk 0 of the V tile row, in the swizzle's place
    const uint32_t dst0 = smem_u32(smem + S::kOffV) + (vpos >> 3) * 1024 + (vpos & 7) * 128 + ((vpos & 7) << 4);
    int first = 0;  // the segment's first block
    int st = w;     // this block's stage
    uint32_t raw_par = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int ms = k % kSegs;
      if (!wwait(&bars.seg_full[ms], static_cast<uint32_t>(k / kSegs) & 1u)) break;
      const int n = segs[ms].n;
      if (n < 0) break;
      const int past = segs[ms].p0 + segs[ms].ntok - segs[ms].j0 * kBS;  // keys of the segment that any row sees
      for (int g = first + ((w ^ first) & 1); g < first + n; g += 2) {
        if (!(ok = wwait(&bars.raw_full[st], raw_par))) break;
        RawRow rk, rv;
        load_row_at(at_k, st * kStageBytes, rk);
        if (!(ok = wwait(&bars.s_out[w], (static_cast<uint32_t>(g >> 1) & 1u) ^ 1u))) break;  // S^T(g - 2)
        tc_fence_after();
#pragma unroll
        for (int qd = 0; qd < 4; ++qd) {  // each quarter goes to TMEM while the next is dequantised
          uint32_t u[8];
          dequant_quarter(rk, qd, lut32, u);
          tmem_st8(tk + 8 * qd, u);
        }
        load_row_at(at_v, st * kStageBytes, rv);
        if ((g - first) * kBS + key_v >= past) {  // after the last position: anything may stand there, 0 x NaN is NaN
          rv.c[0] = rv.c[1] = rv.c[2] = rv.c[3] = make_uint4(0u, 0u, 0u, 0u);
          rv.sc = make_uint2(0u, 0u);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.s_in[w]);
        if (!(ok = wwait(&bars.pv_out[g & 3], (static_cast<uint32_t>(g >> 2) & 1u) ^ 1u))) break;  // block g - 4
        const uint32_t vt = dst0 + (g & 3) * S::kVTile;
#pragma unroll
        for (int qd = 0; qd < 4; ++qd) {
          uint32_t u[8];
          dequant_quarter(rv, qd, lut32, u);
          sts128_at(vt ^ ((2 * qd) << 4), u[0], u[1], u[2], u[3]);
          sts128_at(vt ^ ((2 * qd + 1) << 4), u[4], u[5], u[6], u[7]);
        }
        fence_proxy_async_smem();  // the V tile is read by the tensor core
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars.raw_empty[st]);  // once the rows have been used, not merely loaded
          mbar_arrive(&bars.pv_in[g & 3]);
        }
        st += 2;
        if (st >= S::kStages) {
          st -= S::kStages;
          raw_par ^= 1u;
        }
      }
      first += n;
      if (ok && lane == 0) mbar_arrive(&bars.seg_empty[ms]);
    }
  } else if (warp >= kWarpSm) {
    // ---- softmax warpgroup x: blocks g with g % 2 == x ---------------------------------------------
    const int x = (warp - kWarpSm) >> 2, q = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
    const int hb = 2 * (lane & 3);  // this thread's heads of a token: hb, hb + 1, hb + 8, hb + 9 (slot hh)
    // P^T row (part u of head h: u kN + h) is 128 keys, 128 B; rows n sit at (n / 8) KB + (n % 8) x 128 B. This
    // thread's word (key positions 32 q + 4 (lane / 4) .. + 3) is in chunk 2 q + lane / 16, swizzled by n % 8
    const int pch = 2 * q + (lane >> 4), pb = 4 * ((lane >> 2) & 3);
    uint8_t* pt = smem + S::kOffP;
    uint8_t* const pw0 = pt + hb * 128 + ((pch ^ hb) << 4) + pb;
    uint8_t* const pw1 = pt + (hb + 1) * 128 + ((pch ^ (hb + 1)) << 4) + pb;
    const float c = p.scale_log2;
    float* redm = reinterpret_cast<float*>(smem + S::kOffMax) + x * 4 * kN;
    float* cfs = reinterpret_cast<float*>(smem + S::kOffCf) + x * kN;
    const int bar_vote = kBarVote + x, bar_x = kBarX + x;
    int first = 0;  // the segment's first block
    bool ok = true;
    if (lane == 0) mbar_arrive(&bars.s_in[x]);  // the score slot is free
    // A warp leaves at a vote only, so that its warpgroup's named barriers always find all four.
    for (int k = 0;; ++k) {
      const int ms = k % kSegs;
      const bool got = ok && wwait(&bars.seg_full[ms], static_cast<uint32_t>(k / kSegs) & 1u);
      if (named_barrier_or(bar_vote, 128, !got)) break;
      const Seg& m = segs[ms];
      const int n = m.n;
      if (n < 0) break;
      float ref[4], l[4];
#pragma unroll
      for (int hh = 0; hh < 4; ++hh) ref[hh] = l[hh] = 0.f;
      bool quit = false;
      const int g0 = first + ((x ^ first) & 1);  // this warpgroup's first block of the segment
      for (int g = g0; g < first + n; g += 2) {
        const int base = (m.j0 + g - first) * kBS;
        float d[4][4];  // [key i][head slot hh]: exponents s c - ref
        ok = ok && wwait(&bars.s_out[x], static_cast<uint32_t>(g >> 1) & 1u);
        tc_fence_after();
        uint32_t ra[8], rb[8];
        tmem_ld16x256_x2(tmem + lanes + S::kColS + kN * x, ra);
        tmem_ld16x256_x2(tmem + lanes + (16u << 16) + S::kColS + kN * x, rb);
        tmem_wait_ld();
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            fma_f32x2(__uint_as_float(ra[4 * o + 2 * e]), __uint_as_float(ra[4 * o + 2 * e + 1]), c, c, -ref[2 * o],
                      -ref[2 * o + 1], d[e][2 * o], d[e][2 * o + 1]);
            fma_f32x2(__uint_as_float(rb[4 * o + 2 * e]), __uint_as_float(rb[4 * o + 2 * e + 1]), c, c, -ref[2 * o],
                      -ref[2 * o + 1], d[2 + e][2 * o], d[2 + e][2 * o + 1]);
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.s_in[x]);
        if (base + kBS - 1 > m.p0) {  // keys after a token's position get P = 0
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (base + 32 * q + kappa((lane >> 2) + 8 * i) > m.p0) {
#pragma unroll
              for (int hh = 0; hh < 4; ++hh) d[i][hh] = -CUDART_INF_F;
            }
        }
        float top = d[0][0];
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max3f(max3f(top, d[i][0], d[i][1]), d[i][2], d[i][3]);
        const bool need = top > kRescaleLog2;
        if (g == g0 || named_barrier_or(bar_vote, 128, need || !ok)) {
          if (named_barrier_or(bar_x, 128, !ok || *abort_flag != 0)) {  // a give-up, decided alike in all four
            quit = true;
            break;
          }
          // ---- the references move to this block's maxima less kUp, where those are larger
#pragma unroll
          for (int hh = 0; hh < 4; ++hh) {
            float bm = fmaxf(fmaxf(d[0][hh], d[1][hh]), fmaxf(d[2][hh], d[3][hh])) + ref[hh];
            bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 4));
            bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 8));
            bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 16));
            if (lane < 4) redm[q * kN + hb + (hh & 1) + 8 * (hh >> 1)] = bm;
          }
          named_barrier(bar_x, 128);
#pragma unroll
          for (int hh = 0; hh < 4; ++hh) {
            const int h = hb + (hh & 1) + 8 * (hh >> 1);
            const float bx = fmaxf(fmaxf(redm[h], redm[kN + h]), fmaxf(redm[2 * kN + h], redm[3 * kN + h])) - kUp;
            float to = g == g0 ? bx : fmaxf(ref[hh], bx);
            if (!(to > -CUDART_INF_F)) to = ref[hh];  // no key of the block is visible: keep it finite
            const float cf = g == g0 ? 0.f : fast_exp2(ref[hh] - to);
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i][hh] += ref[hh] - to;
            l[hh] *= cf;
            ref[hh] = to;
            if (q == 0 && lane < 4) cfs[h] = cf;
          }
          named_barrier(bar_x, 128);
          // O^T *= cf once block g - 2 is in it (this thread's lane = dim 32 q + lane)
          if (g > g0) {
            ok = ok && wwait(&bars.pv_out[(g - 2) & 3], static_cast<uint32_t>((g - 2) >> 2) & 1u);
            tc_fence_after();
#pragma unroll 1
            for (int h8 = 0; h8 < kParts * kN; h8 += 8) {  // a part's columns, then the next one's
              uint32_t o[8];
              tmem_ld8(tmem + lanes + S::kColO + S::kOStep * x + h8, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * cfs[(h8 + e) & (kN - 1)]);
              tmem_st8(tmem + lanes + S::kColO + S::kOStep * x + h8, o);
            }
            tmem_wait_st();
            tc_fence_before();
          }
        }
        // ---- P = 2^d -> the parts of P^T, once block g - 4 has been read
        ok = ok && wwait(&bars.pv_out[g & 3], (static_cast<uint32_t>(g >> 2) & 1u) ^ 1u);
        const uint32_t tile = (g & 3) * S::kPTile;
#pragma unroll
        for (int hh = 0; hh < 4; ++hh) {
          float pv[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) pv[i] = fast_exp2(d[i][hh]);
          l[hh] += (pv[0] + pv[1]) + (pv[2] + pv[3]);
          // an f16's upper byte is its E5M2 value rounded towards zero, and what is left is exact
          constexpr uint32_t kUpper = 0xFF00FF00u;
          uint32_t r01 = pack_f16x2(pv[0], pv[1]), r23 = pack_f16x2(pv[2], pv[3]);
          uint8_t* pw = ((hh & 1) ? pw1 : pw0) + tile + 1024 * (hh >> 1);
#pragma unroll
          for (int u = 0; u < kParts - 1; ++u) {
            *reinterpret_cast<uint32_t*>(pw + u * kN * 128) = prmt(r01, r23, 0x7531u);
            r01 = sub_f16x2(r01, r01 & kUpper);
            r23 = sub_f16x2(r23, r23 & kUpper);
          }
          *reinterpret_cast<uint32_t*>(pw + (kParts - 1) * kN * 128) = cvt_e5m2x2_f16x2(mul_f16x2(r01, kLastScale2)) |
                                                                           (cvt_e5m2x2_f16x2(mul_f16x2(r23, kLastScale2)) << 16);
        }
        fence_proxy_async_smem();  // P^T is read by the tensor core
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.pv_in[g & 3]);
      }
      if (quit) break;
      // ---- the segment's result: both slots' sums joined; each warpgroup takes eight of the
      // rows, a thread one dim of them
      float* ls = reinterpret_cast<float*>(smem + S::kOffL) + (k & 1) * 2 * 4 * kN;
      float* refs = reinterpret_cast<float*>(smem + S::kOffRef) + (k & 1) * 2 * kN;
#pragma unroll
      for (int hh = 0; hh < 4; ++hh) {
        float s = l[hh];
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        const int h = hb + (hh & 1) + 8 * (hh >> 1);
        if (lane < 4) ls[(x * 4 + q) * kN + h] = s;
        if (lane < 4 && q == 0) refs[x * kN + h] = ref[hh];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bars.ml);
      ok = ok && wwait(bars.ml, static_cast<uint32_t>(k) & 1u);
      {  // the last block's PV, and with it all before
        const int last = first + n - 1;
        ok = ok && wwait(&bars.pv_out[last & 3], static_cast<uint32_t>(last >> 2) & 1u);
      }
      bool used[2];  // a segment of one block fills one slot
#pragma unroll
      for (int y = 0; y < 2; ++y) used[y] = n > 1 || (first & 1) == y;
      first += n;
      tc_fence_after();
      if (ok) {
        const int dim = 32 * q + lane;
        const int h0 = 8 * x;
        float o[2][8];  // the parts added up, one load in flight a slot (all at once would spill)
#pragma unroll
        for (int u = kParts - 1; u >= 0; --u) {
          uint32_t t[2][8];
#pragma unroll
          for (int y = 0; y < 2; ++y)
            if (used[y]) tmem_ld8(tmem + lanes + S::kColO + S::kOStep * y + kN * u + h0, t[y]);
          tmem_wait_ld();
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              o[y][e] = u == kParts - 1 ? __uint_as_float(t[y][e]) * (1.f / kLastScale) : o[y][e] + __uint_as_float(t[y][e]);
        }
        const bool bad = m.bad <= m.p0;
        // lane e works out row h0 + e (mod 8): its sum, and what each slot's part is multiplied by
        float wy[2], M = -CUDART_INF_F, L = 0.f;
        {
          const int h = h0 + (lane & 7);
          float my[2], ly[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float* a = ls + 4 * y * kN + h;
            ly[y] = used[y] ? (a[0] + a[kN]) + (a[2 * kN] + a[3 * kN]) : 0.f;
            my[y] = ly[y] == 0.f ? -CUDART_INF_F : refs[y * kN + h];  // a slot none of whose keys the row sees: sum 0
            M = fmaxf(M, my[y]);
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            wy[y] = ly[y] == 0.f ? 0.f : fast_exp2(my[y] - M);
            L = fmaf(wy[y], ly[y], L);
          }
          if (m.part < 0) {
            const float inv = bad ? 0.f : 1.f / L;
            wy[0] *= inv;
            wy[1] *= inv;
            if (p.lse != nullptr && q == 0 && lane < 8)
              p.lse[static_cast<int64_t>(m.t0) * kQHeads + m.g * kHPG + h] =
                  bad ? -CUDART_INF_F : (M + __log2f(L)) * 0.69314718055994531f;
          } else if (q == 0 && lane < 8) {
            p.part_ml[(static_cast<int64_t>(blockIdx.x) * 2 + m.part) * kN + h] =
                make_float2(bad ? CUDART_NAN_F : M, L);
          }
        }
        const int64_t orow = static_cast<int64_t>(m.t0) * kQHeads + m.g * kHPG + h0;
        const int64_t prow = (static_cast<int64_t>(blockIdx.x) * 2 + m.part) * kN + h0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float v = 0.f;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float w = __shfl_sync(0xffffffffu, wy[y], e);
            if (w != 0.f)
              v = fmaf(w, o[y][e], v);
          }
          if (m.part < 0) reinterpret_cast<__nv_bfloat16*>(p.out)[(orow + e) * kD + dim] = __float2bfloat16_rn(v);
          else p.part_o[(prow + e) * kD + dim] = v;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bars.o_free);
        mbar_arrive(&bars.seg_empty[ms]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpTmem) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

}  // namespace few

// Joins the parts of the (tile, group) that starts in span blockIdx.x and ends in a later one: its
// first part is that span's second place, the others the following spans' first places. Up to eight
// parts: a warp a row, lane = 4 dims, four loads in flight. More (few rows, long contexts): a CTA a row,
// the parts' weights by all threads, their sums by the eight warps in turn, added in a fixed order. (A
// warp a row for 32 parts took 21 us; a CTA a row for the 128 rows of 2 parts of 128 tiles 35 us more
// than a warp.) A part on a bad page (reference NaN) makes the row zero.
__global__ void __launch_bounds__(256) k_dense_join(const DenseParams p) {
  __shared__ float wt[kSpans + 1];
  __shared__ float4 acc[8][32];
  __shared__ float red[2][8];
  grid_dependency_wait();
  const int4 rec = p.rec[blockIdx.x];
  const int parts = rec.x, rows = rec.z * kHPG, tile_rows = p.tile_tok * kHPG;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (parts < 2) return;
  if (parts <= 8) {
    const int r = blockIdx.y * 8 + warp;
    if (r >= rows) return;
    auto place = [&](int i) {
      return (static_cast<int64_t>(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * tile_rows + r;
    };
    const float2 ml = lane < parts ? p.part_ml[place(lane)] : make_float2(-CUDART_INF_F, 0.f);
    float4 v[4];  // the first parts' sums load while their weights are worked out
    auto load = [&](int i) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        v[u] = i + u < parts ? *reinterpret_cast<const float4*>(p.part_o + place(i + u) * kD + 4 * lane)
                             : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    load(0);
    const bool bad = __any_sync(0xffffffffu, ml.x != ml.x);
    float M = ml.x;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    M = __shfl_sync(0xffffffffu, M, 0);
    const float w = ml.x == -CUDART_INF_F ? 0.f : fast_exp2(ml.x - M);
    float L = w * ml.y;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    L = __shfl_sync(0xffffffffu, L, 0);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < parts; i += 4) {
      if (i > 0) load(i);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float wu = __shfl_sync(0xffffffffu, w, i + u);
        if (wu != 0.f) {  // a part none of whose keys the row sees may hold anything
          a.x = fmaf(wu, v[u].x, a.x);
          a.y = fmaf(wu, v[u].y, a.y);
          a.z = fmaf(wu, v[u].z, a.z);
          a.w = fmaf(wu, v[u].w, a.w);
        }
      }
    }
    const int64_t orow = static_cast<int64_t>(rec.y + (r >> 4)) * kQHeads + rec.w * kHPG + (r & 15);
    const float inv = bad ? 0.f : 1.f / L;
    *reinterpret_cast<uint2*>(p.out + orow * kD + 4 * lane) =
        bad ? make_uint2(0u, 0u) : make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
    if (p.lse != nullptr && lane == 0) p.lse[orow] = bad ? -CUDART_INF_F : (M + __log2f(L)) * 0.69314718055994531f;
    return;
  }
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    auto place = [&](int i) {
      return (static_cast<int64_t>(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * tile_rows + r;
    };
    // parts <= kSpans < 256: a thread a part
    const float2 ml = tid < parts ? p.part_ml[place(tid)] : make_float2(-CUDART_INF_F, 0.f);
    float4 v[4];
    auto load = [&](int i) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        v[u] = i + 8 * u < parts ? *reinterpret_cast<const float4*>(p.part_o + place(i + 8 * u) * kD + 4 * lane)
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    load(warp);
    const bool bad = __syncthreads_or(ml.x != ml.x);
    float M = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) red[0][warp] = M;
    __syncthreads();
    M = red[0][0];
#pragma unroll
    for (int w = 1; w < 8; ++w) M = fmaxf(M, red[0][w]);
    const float w = ml.x == -CUDART_INF_F ? 0.f : fast_exp2(ml.x - M);
    if (tid < parts) wt[tid] = w;
    float l = w * ml.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) red[1][warp] = l;
    __syncthreads();
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = warp; i < parts; i += 32) {
      if (i > warp) load(i);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float wu = i + 8 * u < parts ? wt[i + 8 * u] : 0.f;
        if (wu != 0.f) {  // a part none of whose keys the row sees may hold anything
          a.x = fmaf(wu, v[u].x, a.x);
          a.y = fmaf(wu, v[u].y, a.y);
          a.z = fmaf(wu, v[u].z, a.z);
          a.w = fmaf(wu, v[u].w, a.w);
        }
      }
    }
    acc[warp][lane] = a;
    __syncthreads();
    if (tid < kD) {
      const float* f = reinterpret_cast<const float*>(acc);
      float v = 0.f, L = 0.f;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        v += f[x * kD + tid];
        L += red[1][x];
      }
      const int64_t orow = static_cast<int64_t>(rec.y + (r >> 4)) * kQHeads + rec.w * kHPG + (r & 15);
      reinterpret_cast<__nv_bfloat16*>(p.out)[orow * kD + tid] = __float2bfloat16_rn(bad ? 0.f : v / L);
      if (p.lse != nullptr && tid == 0) p.lse[orow] = bad ? -CUDART_INF_F : (M + __log2f(L)) * 0.69314718055994531f;
    }
    __syncthreads();
  }
}

// Tokens a tile: 16 (two row tiles, K and V dequantised once for both) where a sequence may hold
// more than 8, else 8; 1 (k_dense_few) where none holds more. Both sides, 32 sequences of 16K: one token 75 us
// with k_dense_few and 98 with tiles of 8, two tokens 128 and 100; nine tokens 160 us with tiles of 16 and 198
// with tiles of 8, 32 tokens 322 and 386; a 2,048-token prompt at 16K 563 and 680. The rule is the batch's, not a
// sequence's: 31 sequences of one token at 32K take 127 us by themselves, 173 with tiles of 8 and 189 with tiles of 16,
// and in one batch with a 2,048-token chunk at 16K 826 us, where the two calls take 692.
int tile_log2(int32_t max_q_len) { return max_q_len > kTileTok ? 4 : (max_q_len > 1 ? 3 : 0); }

// Scores of |z| up to 2^24 keep their row: an exponent's reference is then rounded to 1, so that the largest P is
// within a factor of 2 of where it should lie, inside f16. The smallest product of two E4M3 values but 0 is 2^-18, so
// that a larger scale has no other score in that range, and 3e38 x log2(e) is infinite.
constexpr float kMostScale = 0x1p42f;

struct Layout {
  size_t rec, ml, o, total;
};
Layout dense_layout(int32_t max_q_len) {
  using msa_host::align256;
  const size_t rows = static_cast<size_t>(kSpans) * 2 * (kHPG << tile_log2(max_q_len));
  Layout w;
  w.rec = 0;
  w.ml = align256(kSpans * sizeof(int4));
  w.o = w.ml + align256(rows * sizeof(float2));
  w.total = w.o + rows * kD * sizeof(float);
  return w;
}

}  // namespace
}  // namespace msa

using namespace msa;
using namespace msa_host;

extern "C" size_t msa_dense_attn_workspace_size(const msa_geometry* geo, int32_t B, int32_t T, int32_t max_q_len) {
  if (check_geometry(geo) != MSA_OK || B < 0 || B > 4096 || T < 0 || T > (1 << 22) || max_q_len < 1 ||
      max_q_len > (1 << 20))
    return 0;
  return dense_layout(max_q_len).total;
}

extern "C" msa_status msa_dense_attn(const msa_geometry* geo, const msa_batch* batch, const msa_cache* cache,
                                     const uint8_t* q, float softmax_scale, void* workspace, size_t workspace_bytes,
                                     uint16_t* out, float* lse, uint32_t* status, cudaStream_t stream) {
  msa_status st = check_geometry(geo);
  if (st != MSA_OK) return st;
  if ((st = check_prefill_batch(batch)) != MSA_OK) return st;
  if ((st = check_cache(cache, false, true)) != MSA_OK) return st;
  if (!(softmax_scale > 0.0f) || !(softmax_scale <= kMostScale)) return MSA_ERR_INVALID_ARG;
  if (batch->B == 0 || batch->T == 0) return MSA_OK;
  if (q == nullptr || out == nullptr || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || cache->num_pages == 0)
    return MSA_ERR_INVALID_ARG;
  const Layout w = dense_layout(batch->max_q_len);
  if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < w.total) return MSA_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const DenseParams p{batch->B, batch->T, batch->max_blocks_per_seq, batch->max_q_len, cache->num_pages,
                      1 << tile_log2(batch->max_q_len), tile_log2(batch->max_q_len), batch->query_start_loc, batch->seq_lens, batch->block_table,
                      softmax_scale * 1.4426950408889634f, out, lse, status, reinterpret_cast<int4*>(ws + w.rec),
                      reinterpret_cast<float*>(ws + w.o), reinterpret_cast<float2*>(ws + w.ml)};
  alignas(64) CUtensorMap kv_map, q_map;
  if (!kv_tensor_map(&kv_map, cache->kv_pages, static_cast<uint64_t>(cache->num_pages)) ||
      !rows128_tensor_map(&q_map, q, static_cast<uint64_t>(batch->T) * kQHeads, kHPG))
    return MSA_ERR_CUDA;
  void (*kernel)(DenseParams, CUtensorMap, CUtensorMap) = p.tile_tok > kTileTok ? k_dense<true> : k_dense<false>;
  int threads = kThreads;
  size_t smem = Smem::kBytes;
  if (p.tile_tok == 1) {
    kernel = few::k_dense_few;
    threads = few::kThreads;
    smem = few::Sm::kBytes;
  }
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
    return MSA_ERR_CUDA;
  // both kernels set up while the one before them on the stream ends, and wait for it before they read
  if (launch_after_previous(kernel, dim3(kSpans), dim3(threads), smem, stream, p, kv_map, q_map) != cudaSuccess)
    return MSA_ERR_CUDA;
  const int rows = p.tile_tok * kHPG;
  if (launch_after_previous(k_dense_join, dim3(kSpans, rows < 32 ? rows : 32), dim3(256), 0, stream, p) != cudaSuccess)
    return MSA_ERR_CUDA;
  return launch_status();
}
