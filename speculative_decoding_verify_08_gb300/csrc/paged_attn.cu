// paged_attn.cu -- attention of the newest M rows of each of B sequences over
// a paged cache (M = 1: one new token), with an optional sliding window and a
// few first tokens that stay visible.
//
// Row i of sequence b stands at position p = len_b - M + i and sees position
// j iff j <= p and (no window, or j > p - window, or j < sinks):
//   O = softmax_j(scale <Q, K_j>) V,   zeros where nothing is seen.
//
// What bounds it: every visible slot of K and V is read once and meets
// M*Hq/Hkv query rows, so HBM (and, for short sequences, latency).  Hence:
//  * The work of a call is a line of units, one unit a 16-slot chunk of one
//    (sequence, KV head); only chunks that some row sees are on it, and each
//    (sequence, head) begins with HEAD_COST more for what it costs beside its
//    chunks (queries, join, output).  Every CTA (one per SM) finds the line's
//    length from the device's lengths and takes an equal, contiguous piece, so
//    ragged batches and long single sequences load all SMs alike and the host
//    needs no lengths.  Where heads are few, each is cut into equal pieces of
//    its own instead, so that no CTA has two, if these are no longer than the
//    line's.
//  * Four producer warps stream chunks into a shared-memory ring by TMA, one
//    5-D copy for K and one for V (page, head, 64-column group, slot, column),
//    looking pages up 32 chunks ahead.  A chunk never crosses a page.  (A copy
//    and the wait before it keep a warp for about 250 ns, longer than a chunk's
//    share of HBM: hence four.  Waiting for several chunks' slots before their
//    copies costs more than it hides: 119 -> 129 us for 200000 slots of 4 x 256.)
//  * Each of eight consumer warps takes every (8/MT)-th chunk for one 16-row
//    tile of query rows and keeps its own running maximum, sum and O in
//    registers: the scores' accumulator layout is the next product's operand
//    layout, so nothing but the ring is shared and no barrier stands in the
//    loop.  The warps' results are joined once per (sequence, head).
//  * A piece that does not hold all of its (sequence, head) leaves its O,
//    maximum and sum in the workspace; a second kernel joins them.
//  * The maximum is raised only when a chunk exceeds it by more than 2^8 (2^2
//    beside an e4m3 cache), so the accumulators are rarely rescaled.
// Probabilities are rounded to the operand type of the second product, one
// rounding each.  bf16: relative 2^-8 whatever their size.  fp16 (beside an
// e4m3 cache, whose values it holds exactly): relative 2^-11 in its normal
// range only, so they are taken 2^13 times as large, up to 2^15 of 65504, and
// the sum with them, so that the factor cancels: those down to 2^-27 of the
// maximum keep 2^-11, smaller ones are off by 2^-38 of the maximum at most
// (against 1 for the maximum, many small ones beside a large one lost 2^-25
// each, up to all of their share).
// An e4m3 cache is converted in registers to fp16; the queries are scaled by a
// power of two per row to fit fp16: exact down to 2^-14 of a row's largest
// element, off by 2^-25 of that below.
// Measured, as calls: 48 sequences of 40 to 16000 slots, 32/8 heads of 128: 96 us,
// 6.2 TB/s; 64 with a window of 4096 on 16 heads: 306 us, 6.7 TB/s; one of 32768, 4
// rows, 24/4 heads of 256: 28.8 us (27.2 on the GPU), 4.7 TB/s (start and join of
// a short stream); one of 777: 9.0 us (8.8); over e4m3 pages, 24 of 500 to 32000,
// 24/4 heads of 256: one row 89 us, 5.7 TB/s; 4 rows 135 us, 3.7 TB/s, held back by
// the conversions, which both 16-row tiles' warps make.
#include <cstring>

#include "paged.cuh"

namespace sv {
namespace attn {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // attn.cu
}
namespace paged {

constexpr int CHUNK = 16;  // slots per unit
constexpr int NCW = 8;     // consumer warps
constexpr int NPW = 4;     // producer warps: K and V of even and odd chunks
constexpr int THREADS = (NCW + NPW) * 32;
// 384 threads start with 168 registers each; 128 * 72 + 256 * 216 is the same total
constexpr int REGS_PRODUCER = 72, REGS_CONSUMER = 216;
constexpr int MAX_B = 4096;
constexpr int MAX_R = 128;           // query rows per KV head: eight 16-row tiles
constexpr int MAX_STAGES = 32;
constexpr int HEAD_COST = 12;        // chunks' time that a (sequence, head) takes beside its chunks
constexpr int MAX_EVEN_B = 64;       // sequences up to which heads are cut evenly
// log2 of the factor on probabilities and their sum, and of the largest
// probability, factor included, before the maximum is raised
__host__ __device__ constexpr float lift(bool f8) { return f8 ? 13.f : 0.f; }
__host__ __device__ constexpr float largest(bool f8) { return f8 ? 15.f : 8.f; }
constexpr size_t SMEM_LIMIT = 227 * 1024;

struct Params {
  sv_rows q, o;
  const int *table;
  long long table_stride;
  int width;  // pages per table row
  const int *lens;
  const float *ks, *vs;
  float *opart;  // [2 * ctas][R][D] unnormalised O
  float *ml;     // [2 * ctas][R][2] maximum (log2 domain) and sum
  int4 *desc;    // [ctas] split heads: (b * Hkv + h, first CTA, CTAs, -)
  unsigned *err;
  int B, M, Hkv, G, R;
  float sl2e;  // scale * log2(e)
  int window, sinks;
  int page_size, num_pages;
  int stages;
  int min_units;  // least units per CTA
  int by_head;    // desc is indexed by b * Hkv + h (else by CTA)
  int stall;      // test aid: the ring's first slot never fills
};

// Chunks of one sequence that some row sees: the first `ns` chunks, then
// chunks w0..ce-1.
struct Span {
  int L, ns, w0, ce;
  __device__ __forceinline__ int count() const { return ns + ce - w0; }
  __device__ __forceinline__ int chunk(int k) const { return k < ns ? k : k - ns + w0; }
};

__device__ __forceinline__ int first_seen(const Params &P, int L) {
  return P.window > 0 ? imax(0, L - P.M - P.window + 1) : 0;
}

__device__ __forceinline__ Span span_of(const Params &P, int L) {
  Span s;
  s.L = L;
  s.ce = (L + CHUNK - 1) / CHUNK;
  s.w0 = first_seen(P, L) / CHUNK;
  s.ns = (imin(P.sinks, L) + CHUNK - 1) / CHUNK;
  if (s.w0 <= s.ns) s.w0 = s.ns = 0;
  return s;
}

__device__ __forceinline__ int length_of(const Params &P, int b) {
  const long long cap = (long long)P.width * P.page_size;
  const int l = P.lens[b];
  if (l < 0 || l > cap) {
    if (blockIdx.x == 0) atomicOr(P.err, ERR_INDEX);
    return l < 0 ? 0 : (int)cap;
  }
  return l;
}

// Byte offset of 16-byte group c in row r of a 16-row tile stored as
// 128-byte-wide swizzled boxes.
__device__ __forceinline__ uint32_t swz16(int r, int c) {
  return (uint32_t)((c >> 3) * 2048 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {  // low 16 bits
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}\n" : "=r"(d) : "r"(v));
  return d;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2_hi(uint32_t v) {  // high 16 bits
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}\n" : "=r"(d) : "r"(v));
  return d;
}

template <bool F8>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F8)
    mma_f16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
  else
    mma_bf16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
}

// Ring slots of n chunks that are taken N at a time.
template <int N>
__host__ __device__ constexpr int padded(int n) { return (n + N - 1) / N * N; }

template <int D, bool F8, int MT>
struct Layout {
  // Chunks that a consumer warp takes at a time.  Two need twice the ring: one
  // set in work, one under way.
  static constexpr int NCH = F8 && MT > 1 ? 2 : 1;
  static constexpr int TILE = CHUNK * D * (F8 ? 1 : 2);  // bytes of a chunk of K (or V)
  static constexpr int STAGE = 2 * TILE;
  static constexpr int QS = 1024;                         // after the barriers
  static constexpr int QBYTES = MT * 16 * D * 2;
  static constexpr int RS = F8 ? D + 16 : D + 8;          // scratch row stride, floats: no bank met twice
  static constexpr int SCRATCH = QS + QBYTES;
  static constexpr int SBYTES = NCW * 8 * RS * 4;
  static constexpr int ML = SCRATCH + SBYTES;             // [NCW][16][2] floats
  static constexpr int FIN = ML + NCW * 16 * 8;           // [MT*16][2] floats
  static constexpr int QSC = FIN + MT * 16 * 8;           // [MT*16] floats
  static constexpr int RING = (QSC + MT * 16 * 4 + 1023) / 1024 * 1024;
  // the prefix sums (B + 1 ints) follow the ring
};

template <int D, bool F8, int MT>
__global__ void __launch_bounds__(THREADS, 1)
    paged_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                 const Params P) {
  using LY = Layout<D, F8, MT>;
  constexpr int NL = NCW / MT;  // warps that take turns
  constexpr int NCH = LY::NCH;
  constexpr int NKS = D / 16;
  constexpr int NT = D / 8;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem);
  uint64_t *empty = full + MAX_STAGES;
  int *wsum = reinterpret_cast<int *>(smem + 512);  // scan: warp totals
  int *cuts = reinterpret_cast<int *>(smem + 640);  // even cuts: pieces before sequence b, per head
  uint8_t *qs = smem + LY::QS;
  float *scratch = reinterpret_cast<float *>(smem + LY::SCRATCH);
  float *sml = reinterpret_cast<float *>(smem + LY::ML);
  float *fin = reinterpret_cast<float *>(smem + LY::FIN);
  float *qsc = reinterpret_cast<float *>(smem + LY::QSC);
  uint8_t *ring = smem + LY::RING;
  const int NST = P.stages;
  int *pre = reinterpret_cast<int *>(ring + NST * LY::STAGE);  // pre[b]: units before sequence b, per head

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < NST) {
    mbar_init(&full[tid], 2 + (tid == 0 ? P.stall : 0));  // K and V
    mbar_init(&empty[tid], MT);
    fence_barrier_init();
  }
  pdl_wait();

  // ---- the line of units: prefix sums of the sequences' costs ----
  int total = 0;
  for (int b0 = 0; b0 < P.B; b0 += THREADS) {
    const int b = b0 + tid;
    const int chunks = b < P.B ? span_of(P, length_of(P, b)).count() : 0;
    const int n = chunks > 0 ? chunks + HEAD_COST : 0;
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += wsum[w];
      all += wsum[w];
    }
    if (b < P.B) pre[b] = total + before + x - n;
    total += all;
    __syncthreads();
  }
  if (tid == 0) pre[P.B] = total;
  __syncthreads();

  const int units = total * P.Hkv, ctas = (int)gridDim.x;
  const int per = imax(P.min_units + HEAD_COST, (int)(((unsigned)units + (unsigned)ctas - 1) / (unsigned)ctas));
  const int u0 = (int)lmin(units, (long long)per * blockIdx.x), u1 = (int)lmin(units, (long long)u0 + per);

  // ---- even cuts, where heads are few: the shortest piece length for which
  // the pieces are no more than the CTAs (every warp works it out) ----
  bool even = false;
  if (P.by_head && P.B <= MAX_EVEN_B) {
    auto chunks_of = [&](int b) { return b < P.B ? imax(0, pre[b + 1] - pre[b] - HEAD_COST) : 0; };
    const int n0 = chunks_of(lane), n1 = chunks_of(lane + 32);
    const int all = __reduce_add_sync(0xffffffffu, n0 + n1) * P.Hkv;
    int len = imax(P.min_units, (all + ctas - 1) / ctas), pieces = 0;
    auto cut = [&]() {
      pieces = (n0 + len - 1) / len + (P.B > 32 ? (n1 + len - 1) / len : 0);
      return __reduce_add_sync(0xffffffffu, pieces) * P.Hkv;
    };
    // longer at every step by half the share that the last one overshot
    int x = cut();
    while (x > ctas && len <= per) {
      len += 1 + (int)((float)len * (float)(x - ctas) / (float)(2 * ctas));
      x = cut();
    }
    even = x <= ctas && len <= per;
    if (even && warp == 0) {
      int x0 = (n0 + len - 1) / len, x1 = (n1 + len - 1) / len;
      const int own0 = x0, own1 = x1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y0 = __shfl_up_sync(0xffffffffu, x0, o), y1 = __shfl_up_sync(0xffffffffu, x1, o);
        if (lane >= o) x0 += y0, x1 += y1;
      }
      const int first32 = __shfl_sync(0xffffffffu, x0, 31);
      cuts[lane] = x0 - own0;
      cuts[lane + 32] = first32 + x1 - own1;
      if (lane == 31) cuts[64] = first32 + x1;
    }
  }
  __syncthreads();

  // sequence of unit u < units
  auto seq_of = [&](int u) {
    const int c = u / P.Hkv;  // chunk-line position rounded down: same sequence as u
    int lo = 0, hi = P.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= c) lo = mid; else hi = mid - 1;
    }
    return lo;  // the last sequence that starts at or before c, so it is not empty
  };
  // The pieces of this CTA, one after the other: chunks ka..kb-1 of n of (b, h);
  // `count`: the pieces of the head, which lie in consecutive CTAs.
  struct Piece {
    int u, b, b0, h, n, ka, kb, count;  // b0: the piece's sequence; b: where the search goes on
  };
  auto start = [&]() {
    Piece x{};
    x.u = even ? 0 : u0;
    x.b = !even && u0 < u1 ? seq_of(u0) : 0;
    return x;
  };
  auto next = [&](Piece &x) {
    if (even) {
      if (x.u > 0) return false;
      x.u = 1;
      const int c = blockIdx.x;
      if (c >= cuts[P.B] * P.Hkv) return false;
      while (cuts[x.b + 1] * P.Hkv <= c) ++x.b;
      const int in = c - cuts[x.b] * P.Hkv;
      x.count = cuts[x.b + 1] - cuts[x.b];
      x.h = in / x.count;
      const int i = in - x.h * x.count;
      x.n = pre[x.b + 1] - pre[x.b] - HEAD_COST;
      x.ka = (int)((long long)x.n * i / x.count);
      x.kb = (int)((long long)x.n * (i + 1) / x.count);
      x.b0 = x.b;
      return true;
    }
    while (x.u < u1) {
      while (pre[x.b + 1] == pre[x.b]) ++x.b;  // (a unit follows: a non-empty sequence exists)
      const int cost = pre[x.b + 1] - pre[x.b], head0 = pre[x.b] * P.Hkv;
      x.h = (x.u - head0) / cost;
      const int at = head0 + x.h * cost, xa = x.u - at, xb = imin(cost, xa + (u1 - x.u));
      x.n = cost - HEAD_COST;
      x.ka = imax(0, xa - HEAD_COST);
      x.kb = imax(0, xb - HEAD_COST);
      x.u += xb - xa;
      x.count = (at + cost - 1) / per - (at + HEAD_COST) / per + 1;
      x.b0 = x.b;
      if (x.h == P.Hkv - 1 && xb == cost) ++x.b;
      if (x.ka < x.kb) return true;
    }
    return false;
  };

  if (warp >= NCW) {
    // ------------------------------------------------------ producers --
    // Two warps stream K, two V; the pairs take turns chunk by chunk.
    setmaxnreg_dec<REGS_PRODUCER>();
    // A lane works out the page and slot of one chunk of the next 32, so that
    // the chunks' own turns hold little but the wait and the copies.
    const bool is_v = (warp - NCW) & 1;
    const int turn = (warp - NCW) >> 1;
    const uint64_t pol = l2_evict_first_policy();
    const int cpp = P.page_size / CHUNK;
    bool ok = true;
    uint32_t q = 0, parity = 1;
    int slot = 0;
    for (Piece x = start(); ok && next(x);) {
      const int b = x.b0, h = x.h, ka = x.ka, kb = x.kb;
      const Span s = span_of(P, length_of(P, b));
      const int *row = P.table + (long long)b * P.table_stride;
      auto page_at = [&](int k) {
        if (k >= kb) return 0;
        const int pg = row[s.chunk(k) / cpp];
        if ((unsigned)pg >= (unsigned)P.num_pages) atomicOr(P.err, ERR_INDEX);
        return pg;
      };
      int next = page_at(ka + lane);
      const int kp = ka + padded<NCH>(kb - ka);  // the slot that fills up a pair gets no copy
      for (int k0 = ka; k0 < kp && ok; k0 += 32) {
        const int page = next;
        next = page_at(k0 + 32 + lane);
        const int m = imin(32, kp - k0);
        const int at = (s.chunk(imin(k0 + lane, kb - 1)) % cpp) * CHUNK;
        for (int i = 0; i < m; ++i, ++q) {
          if ((int)(q & 1) == turn) {
            const int pg = __shfl_sync(0xffffffffu, page, i), sl = __shfl_sync(0xffffffffu, at, i);
            ok = __all_sync(0xffffffffu, mbar_wait(&empty[slot], parity, P.err));
            if (!ok) break;
            if (lane == 0) {
              if (k0 + i >= kb) {
                mbar_arrive(&full[slot]);
              } else {
                mbar_arrive_expect_tx(&full[slot], LY::TILE);
                // a page out of range reads zeros (the copy is clipped to the cache)
                tma_load_5d(ring + slot * LY::STAGE + (is_v ? LY::TILE : 0), is_v ? &mapV : &mapK, 0, sl, 0, h, pg,
                            &full[slot], pol);
              }
            }
          }
          if (++slot == NST) {
            slot = 0;
            parity ^= 1;
          }
        }
      }
    }
    if (!ok && lane == 0) {  // a wait ran out: no copy may outlive the CTA
      const uint32_t first = q > (uint32_t)NST ? q - NST : 0u;
      for (uint32_t qq = first; qq < q && mbar_wait(&full[qq % NST], (qq / NST) & 1, P.err); ++qq) {
      }
    }
    return;
  }

  // --------------------------------------------------------- consumers --
  setmaxnreg_inc<REGS_CONSUMER>();
  const int mt = warp % MT, cl = warp / MT;  // query tile; which of every NL chunks
  const int gq = lane >> 2, tq = lane & 3;
  const int row0 = 16 * mt + gq, row1 = row0 + 8;
  const int i0 = row0 / P.G, i1 = row1 / P.G;
  bool ok = true;
  uint32_t q0 = 0;  // chunks before this segment

  // outputs and descriptors of empty sequences, shared over the CTAs
  for (int b = blockIdx.x; b < P.B; b += ctas) {
    if (pre[b + 1] != pre[b]) continue;
    const int rows = P.M * P.Hkv * P.G;
    for (int x = tid; x < rows * (D / 8); x += NCW * 32) {
      const int r = x / (D / 8), c = x % (D / 8);
      const int i = r / (P.Hkv * P.G), hq = r % (P.Hkv * P.G);
      *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(P.o.ptr) +
                                 ((long long)b * P.M + i) * P.o.token_stride + hq * P.o.head_stride + 8 * c) =
          make_uint4(0u, 0u, 0u, 0u);
    }
    if (P.by_head)
      for (int h = tid; h < P.Hkv; h += NCW * 32) P.desc[b * P.Hkv + h] = make_int4(0, 0, 0, 0);
  }
  if (!P.by_head && tid == 0) P.desc[blockIdx.x] = make_int4(0, 0, 0, 0);

  for (Piece piece = start(); next(piece);) {
    const int b = piece.b0, h = piece.h, n = piece.n, ka = piece.ka, kb = piece.kb;
    const Span s = span_of(P, length_of(P, b));
    const int L = s.L, p0 = L - P.M;  // position of row 0
    const int lo = first_seen(P, L);

    // ---- query rows of this head: r = i*G + j, 128-byte swizzled ----
    constexpr int QN = MT * 16 * (D / 8) / (NCW * 32);  // 16-byte groups a thread
    constexpr int QB = QN < 4 ? QN : 4;                 // with so many loads in flight
    const __nv_bfloat16 *qb = static_cast<const __nv_bfloat16 *>(P.q.ptr) + (long long)b * P.M * P.q.token_stride +
                              (long long)h * P.G * P.q.head_stride;
#pragma unroll 1
    for (int x0 = tid; x0 < MT * 16 * (D / 8); x0 += QB * NCW * 32) {
      uint4 qv[QB];
#pragma unroll
      for (int k = 0; k < QB; ++k) {
        const int r = (x0 + k * NCW * 32) / (D / 8), c = x0 % (D / 8);
        const int i = r / P.G, j = r - i * P.G;
        qv[k] = r < P.R ? *reinterpret_cast<const uint4 *>(qb + (long long)i * P.q.token_stride +
                                                           (long long)j * P.q.head_stride + 8 * c)
                        : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int k = 0; k < QB; ++k) {
        const int r = (x0 + k * NCW * 32) / (D / 8), c = x0 % (D / 8);
        const uint4 v = qv[k];
        uint8_t *tile = qs + (r >> 4) * 16 * D * 2;
        const int rr = r & 15;
        if (!F8) {
          *reinterpret_cast<uint4 *>(tile + swz16(rr, c)) = v;
        } else {
          // fp16 rows scaled so that the largest element is in [1, 2); within 16
          // elements, 4t..4t+3 go where an e4m3 word's elements meet them
          float f[8] = {bf16lo(v.x), bf16hi(v.x), bf16lo(v.y), bf16hi(v.y),
                        bf16lo(v.z), bf16hi(v.z), bf16lo(v.w), bf16hi(v.w)};
          float mx = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(f[e]));
#pragma unroll
          for (int o = D / 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          int ex = (int)(__float_as_uint(mx) >> 23) - 127;
          if (ex < -126 || ex > 126) ex = ex < 0 ? (mx > 0.f ? -126 : 0) : (ex > 127 ? 0 : 126);
          const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
          if (c == 0) qsc[r] = __uint_as_float((uint32_t)(127 + ex) << 23);
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = pack_f16x2(f[2 * e] * down, f[2 * e + 1] * down);
          // chunk c holds elements 8(c&1).. of its group of 16: t = 2(c&1), 2(c&1)+1
          const int g16 = c & ~1, t = 2 * (c & 1);
          uint32_t *lo16 = reinterpret_cast<uint32_t *>(tile + swz16(rr, g16));
          uint32_t *hi16 = reinterpret_cast<uint32_t *>(tile + swz16(rr, g16 + 1));
          lo16[t] = w[0], hi16[t] = w[1], lo16[t + 1] = w[2], hi16[t + 1] = w[3];
        }
      }
    }
    named_barrier(1, NCW * 32);

    constexpr bool QREG = D == 128;  // D = 256: O alone takes 128 registers
    constexpr int NQR = QREG ? NKS : 1;
    uint32_t qa[NQR][4];
    const uint32_t qtile = smem_u32(qs + mt * 16 * D * 2);
    const int qr = (lane & 7) + 8 * ((lane >> 3) & 1);
    if (QREG) {
#pragma unroll
      for (int ks = 0; ks < NQR; ++ks) ldmatrix_x4(qa[ks], qtile + swz16(qr, 2 * ks + (lane >> 4)));
    }
    float sc0 = P.sl2e, sc1 = P.sl2e;
    if (F8) {
      const float kscale = P.ks ? P.ks[h] : 1.f;
      sc0 *= kscale * qsc[row0];
      sc1 *= kscale * qsc[row1];
    }

    // m0, m1: what the exponents refer to, the running maximum less the lift
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float o[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[nt][j] = 0.f;

    const uint32_t q1 = q0 + (uint32_t)padded<NCH>(kb - ka);
    auto load_q = [&](int ks, uint32_t (&qf)[4]) {
      if (QREG) {
#pragma unroll
        for (int t = 0; t < 4; ++t) qf[t] = qa[QREG ? ks : 0][t];
      } else {
        ldmatrix_x4(qf, qtile + swz16(qr, 2 * ks + (lane >> 4)));
      }
    };
    const int kr = 8 * (lane >> 4) + (lane & 7), kc = (lane >> 3) & 1;       // K fragments: slot, group
    const int vr = 8 * ((lane >> 3) & 1) + (lane & 7), vc = lane >> 4;       // V fragments
    // this warp's first chunks: the least q >= q0 with q / NCH % NL == cl
    uint32_t q = q0 + (uint32_t)(NCH * ((cl - (int)(q0 / NCH % NL) + NL) % NL));
    int at = (int)(q % (uint32_t)NST);  // its ring slot
    uint32_t parity = (q / (uint32_t)NST) & 1;
    for (; q < q1; q += NCH * NL) {
      uint32_t kt[NCH];
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        kt[c] = smem_u32(ring + (at + c) * LY::STAGE);
        if (ok) ok = mbar_wait(&full[at + c], parity, P.err);
      }
      // a limit may run out in some lanes while the phase completes for others
      ok = __all_sync(0xffffffffu, ok);
      const int now = at;
      at += NCH * NL;
      if (at >= NST) {
        at -= NST;
        parity ^= 1;
      }
      if (!ok) continue;
      // ---- S = Q K^T, 16 rows x 16 slots (of each of the chunks) ----
      // one chunk: two sums per tile, of the even and the odd steps (a product
      // waits for the one before it on the same sum)
      float sa[NCH][2][4], sb[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sb[nt][j] = 0.f;
#pragma unroll
          for (int c = 0; c < NCH; ++c) sa[c][nt][j] = 0.f;
        }
#pragma unroll
      for (int kp = 0; kp < NKS / 2; ++kp) {
        uint32_t ka4[NCH][4], kb4[NCH][4], qf[4], qg[4];
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          if (!F8) {
            ldmatrix_x4(ka4[c], kt[c] + swz16(kr, 4 * kp + kc));
            ldmatrix_x4(kb4[c], kt[c] + swz16(kr, 4 * kp + 2 + kc));
          } else {
            uint32_t kf[4];
            ldmatrix_x4(kf, kt[c] + swz16(kr, 2 * kp + kc));
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              ka4[c][2 * t] = e4m3x2_to_f16x2(kf[2 * t]);
              ka4[c][2 * t + 1] = e4m3x2_to_f16x2_hi(kf[2 * t]);
              kb4[c][2 * t] = e4m3x2_to_f16x2(kf[2 * t + 1]);
              kb4[c][2 * t + 1] = e4m3x2_to_f16x2_hi(kf[2 * t + 1]);
            }
          }
        }
        load_q(2 * kp, qf);
        load_q(2 * kp + 1, qg);
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) mma16<F8>(sa[c][nt], qf, ka4[c][2 * nt], ka4[c][2 * nt + 1]);
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
            mma16<F8>(NCH == 1 ? sb[nt] : sa[c][nt], qg, kb4[c][2 * nt], kb4[c][2 * nt + 1]);
      }
      if (NCH == 1) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) sa[0][nt][j] += sb[nt][j];
      }
      // ---- scale, mask ----
      const int k0 = ka + (int)(q - q0);
      int pos[NCH];
      bool whole = true;  // every row sees every slot of the chunks
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        pos[c] = CHUNK * s.chunk(k0 + c);
        whole = whole && k0 + c < kb && pos[c] + CHUNK - 1 <= p0 &&
                (P.window == 0 || pos[c] >= L - P.window || pos[c] + CHUNK <= P.sinks);
      }
      uint32_t any[NCH];  // bit t: some row sees slot t
      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        uint32_t seen0 = 0xFFFFu, seen1 = 0xFFFFu;  // by this thread's rows
        any[c] = 0xFFFFu;
        if (!whole) {
          auto below = [](int n) { return n <= 0 ? 0u : n >= 16 ? 0xFFFFu : (1u << n) - 1u; };  // bits 0..n-1
          auto seen_by = [&](int p) {
            return below(imin(p + 1, L) - pos[c]) &
                   (P.window == 0 ? 0xFFFFu : ~below(p - P.window + 1 - pos[c]) | below(P.sinks - pos[c]));
          };
          const uint32_t real = k0 + c < kb ? 0xFFFFu : 0u;  // not there to fill up a pair
          seen0 = seen_by(p0 + i0) & real;
          seen1 = seen_by(p0 + i1) & real;
          any[c] = below(L - pos[c]) & (~below(lo - pos[c]) | below(P.sinks - pos[c])) & real;
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float v = sa[c][nt][j] * ((j & 2) ? sc1 : sc0);
            if (!whole) v = (((j & 2) ? seen1 : seen0) >> (8 * nt + 2 * tq + (j & 1)) & 1u) ? v : -INFINITY;
            sa[c][nt][j] = v;
            if (j & 2) mx1 = fmaxf(mx1, v); else mx0 = fmaxf(mx0, v);
          }
      }
      // ---- running maximum, raised only by a chunk far above it ----
      if (__any_sync(0xffffffffu, mx0 > m0 + largest(F8) || mx1 > m1 + largest(F8))) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
        const float n0 = fmaxf(m0, mx0 - lift(F8)), n1 = fmaxf(m1, mx1 - lift(F8));
        const float a0 = n0 == -INFINITY ? 1.f : ex2_approx(m0 - n0);
        const float a1 = n1 == -INFINITY ? 1.f : ex2_approx(m1 - n1);
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          o[nt][0] *= a0;
          o[nt][1] *= a0;
          o[nt][2] *= a1;
          o[nt][3] *= a1;
        }
        m0 = n0;
        m1 = n1;
      }
      const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
      uint32_t pa[NCH][4];
#pragma unroll
      for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const float x0 = ex2_approx(sa[c][nt][0] - b0), x1 = ex2_approx(sa[c][nt][1] - b0);
          const float y0 = ex2_approx(sa[c][nt][2] - b1), y1 = ex2_approx(sa[c][nt][3] - b1);
          l0 += x0 + x1;
          l1 += y0 + y1;
          pa[c][2 * nt] = F8 ? pack_f16x2(x0, x1) : pack_bf16x2(x0, x1);
          pa[c][2 * nt + 1] = F8 ? pack_f16x2(y0, y1) : pack_bf16x2(y0, y1);
        }
      // ---- O += P V; what no row sees may hold anything and counts as zero ----
      uint32_t vm[NCH][2];
      if (!whole) {
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          const uint32_t x = any[c] >> (2 * tq);
          vm[c][0] = (x & 1u ? 0xFFFFu : 0u) | (x & 2u ? 0xFFFF0000u : 0u);
          vm[c][1] = (x & 0x100u ? 0xFFFFu : 0u) | (x & 0x200u ? 0xFFFF0000u : 0u);
        }
      }
#pragma unroll
      for (int np = 0; np < (F8 ? NT / 4 : NT / 2); ++np) {
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          uint32_t vf[4];
          ldmatrix_x4_trans(vf, kt[c] + LY::TILE + swz16(vr, 2 * np + vc));
          if (!whole) {
            vf[0] &= vm[c][0];
            vf[1] &= vm[c][1];
            vf[2] &= vm[c][0];
            vf[3] &= vm[c][1];
          }
          if (!F8) {
            mma16<F8>(o[2 * np], pa[c], vf[0], vf[1]);
            mma16<F8>(o[2 * np + 1], pa[c], vf[2], vf[3]);
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // 16 columns: the even ones, then the odd ones
              const uint32_t x = __byte_perm(vf[2 * e], 0u, 0x3120), y = __byte_perm(vf[2 * e + 1], 0u, 0x3120);
              mma16<F8>(o[4 * np + 2 * e], pa[c], e4m3x2_to_f16x2(x), e4m3x2_to_f16x2(y));
              mma16<F8>(o[4 * np + 2 * e + 1], pa[c], e4m3x2_to_f16x2_hi(x), e4m3x2_to_f16x2_hi(y));
            }
          }
        }
      }
      __syncwarp();
      if (lane < NCH) mbar_arrive(&empty[now + lane]);
    }
    q0 = q1;

    // ---- join the warps of each query tile ----
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    // every lane of a quad holds the same maximum once it has been raised
    if (tq == 0) {
      float *w = sml + warp * 32;
      w[gq * 2] = m0;
      w[gq * 2 + 1] = l0;
      w[(gq + 8) * 2] = m1;
      w[(gq + 8) * 2 + 1] = l1;
    }
    named_barrier(1, NCW * 32);
    float w0, w1;
    {
      float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
      for (int c = 0; c < NL; ++c) {
        t0 = fmaxf(t0, sml[(c * MT + mt) * 32 + gq * 2]);
        t1 = fmaxf(t1, sml[(c * MT + mt) * 32 + (gq + 8) * 2]);
      }
      w0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - t0);
      w1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - t1);
      if (cl == 0 && tq == 0) {
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int c = 0; c < NL; ++c) {
          const float *w = sml + (c * MT + mt) * 32;
          const float a = w[gq * 2], d = w[(gq + 8) * 2];
          s0 += a == -INFINITY ? 0.f : ex2_approx(a - t0) * w[gq * 2 + 1];
          s1 += d == -INFINITY ? 0.f : ex2_approx(d - t1) * w[(gq + 8) * 2 + 1];
        }
        fin[row0 * 2] = t0;
        fin[row0 * 2 + 1] = s0;
        fin[row1 * 2] = t1;
        fin[row1 * 2 + 1] = s1;
      }
    }
    const bool starts = ka == 0, ends = kb == n;
    const size_t slot = (size_t)blockIdx.x * 2 + (starts ? 1 : 0);  // of a piece
    const float vscale = F8 && P.vs ? P.vs[h] : 1.f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (half == 1 && P.R <= 8) break;
      // rows 8*half .. 8*half+7 of every tile, scaled to the joint maximum
      float *mine = scratch + (size_t)(warp * 8 + gq) * LY::RS;
      const float w = half ? w1 : w0;
      if (!F8) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          *reinterpret_cast<float2 *>(mine + 8 * nt + 2 * tq) =
              make_float2(o[nt][2 * half] * w, o[nt][2 * half + 1] * w);
      } else {
#pragma unroll
        for (int c = 0; c < NT / 2; ++c)
          *reinterpret_cast<float4 *>(mine + 16 * c + 4 * tq) =
              make_float4(o[2 * c][2 * half] * w, o[2 * c + 1][2 * half] * w, o[2 * c][2 * half + 1] * w,
                          o[2 * c + 1][2 * half + 1] * w);
      }
      named_barrier(1, NCW * 32);
#pragma unroll(MT < 4 ? MT * 2 : 4)
      for (int x = 0; x < MT * 8 * (D / 4) / (NCW * 32); ++x) {
        const int rr = (x * NCW * 32 + tid) / (D / 4), d = (tid % (D / 4)) * 4;
        const int r = 16 * (rr >> 3) + 8 * half + (rr & 7);
        if (r >= P.R) continue;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < NL; ++c) {
          const float4 v = *reinterpret_cast<const float4 *>(
              scratch + (size_t)((c * MT + (rr >> 3)) * 8 + (rr & 7)) * LY::RS + d);
          a.x += v.x;
          a.y += v.y;
          a.z += v.z;
          a.w += v.w;
        }
        if (starts && ends) {
          const float l = fin[r * 2 + 1];
          const float f = l != 0.f ? vscale / l : 0.f;
          const int i = r / P.G, j = r % P.G;
          *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(P.o.ptr) +
                                     ((long long)b * P.M + i) * P.o.token_stride +
                                     (long long)(h * P.G + j) * P.o.head_stride + d) =
              make_uint2(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f));
        } else {
          *reinterpret_cast<float4 *>(P.opart + (slot * P.R + r) * D + d) = a;
          if (d == 0) {
            P.ml[(slot * P.R + r) * 2] = fin[r * 2];
            P.ml[(slot * P.R + r) * 2 + 1] = fin[r * 2 + 1];
          }
        }
      }
      named_barrier(1, NCW * 32);
    }
    // the head's first piece names its pieces
    if (tid == 0 && starts) {
      const int hh = b * P.Hkv + h;
      const int4 d = make_int4(hh, (int)blockIdx.x, ends ? 0 : piece.count, 0);
      if (P.by_head)
        P.desc[hh] = d;
      else if (!ends)
        P.desc[blockIdx.x] = d;
    }
  }
  pdl_launch_dependents();
}

// Join the pieces of the heads that were split.
constexpr int JOIN_THREADS = 256;
constexpr int MAX_CTAS = 256;  // pieces a head can have

__device__ __forceinline__ void store_row(const Params &P, int hh, int r, int col, float4 a, float l) {
  const int b = hh / P.Hkv, h = hh - b * P.Hkv;
  const float f = l != 0.f ? (P.vs ? P.vs[h] : 1.f) / l : 0.f;
  const int i = r / P.G, j = r - i * P.G;
  *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(P.o.ptr) +
                             ((long long)b * P.M + i) * P.o.token_stride +
                             (long long)(h * P.G + j) * P.o.head_stride + col) =
      make_uint2(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f));
}
// slot of piece i of a head that starts in CTA c: the first CTA's second, the others' first
__device__ __forceinline__ size_t piece(int c, int i) { return (size_t)(c + i) * 2 + (i == 0 ? 1 : 0); }

// Few heads, each in many pieces: a block per (head, row); a thread per piece
// works out the weights, then groups of D/4 threads share the pieces' rows,
// the first AHEAD rows of a group under way meanwhile: 40 pieces at D = 256, 80
// at 128, as many as one sequence of four (two) KV heads has.  (4: 28.5 against
// 27.5 us for one of 32768, 11.0 against 10.3 for one of 8000; 16: 27.0 and 10.5,
// but 9.03 against 8.83 for one of 777.)
template <int D>
__global__ void __launch_bounds__(JOIN_THREADS) join_few_kernel(const Params P) {
  constexpr int LPG = D / 4, NG = JOIN_THREADS / LPG, AHEAD = 10;
  __shared__ float4 part[NG][LPG];
  __shared__ float wts[MAX_CTAS], red[2][JOIN_THREADS / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int4 d = P.desc[blockIdx.x];
  const int n = d.z, r = blockIdx.y, tid = threadIdx.x;
  if (n == 0) return;
  const int grp = tid / LPG, c = tid % LPG;
  auto load = [&](int i) {
    return *reinterpret_cast<const float4 *>(P.opart + (piece(d.y, i) * P.R + r) * D + 4 * c);
  };
  float4 v[AHEAD];
#pragma unroll
  for (int k = 0; k < AHEAD; ++k)
    v[k] = grp + k * NG < n ? load(grp + k * NG) : make_float4(0.f, 0.f, 0.f, 0.f);
  float2 x = make_float2(-INFINITY, 0.f);
  if (tid < n) x = *reinterpret_cast<const float2 *>(P.ml + (piece(d.y, tid) * P.R + r) * 2);
  float top = x.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) == 0) red[0][tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < JOIN_THREADS / 32; ++w) top = fmaxf(top, red[0][w]);
  const float w = x.x == -INFINITY ? 0.f : ex2_approx(x.x - top);
  wts[tid] = w;
  float l = w * x.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if ((tid & 31) == 0) red[1][tid >> 5] = l;
  __syncthreads();
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float f, float4 y) {
    a.x = fmaf(f, y.x, a.x);
    a.y = fmaf(f, y.y, a.y);
    a.z = fmaf(f, y.z, a.z);
    a.w = fmaf(f, y.w, a.w);
  };
#pragma unroll
  for (int k = 0; k < AHEAD; ++k)
    if (grp + k * NG < n) add(wts[grp + k * NG], v[k]);
#pragma unroll 4
  for (int i = grp + AHEAD * NG; i < n; i += NG) add(wts[i], load(i));
  part[grp][c] = a;
  __syncthreads();
  if (grp != 0) return;
#pragma unroll
  for (int g = 1; g < NG; ++g) add(1.f, part[g][c]);
  l = 0.f;
#pragma unroll
  for (int k = 0; k < JOIN_THREADS / 32; ++k) l += red[1][k];
  store_row(P, d.x, r, 4 * c, a, l);
}

// Many heads: at most one per CTA is split, most in two pieces.  A group of
// D/4 threads takes a row.
template <int D>
__global__ void __launch_bounds__(JOIN_THREADS) join_many_kernel(const Params P) {
  constexpr int LPG = D / 4, NG = JOIN_THREADS / LPG;
  pdl_wait();
  pdl_launch_dependents();
  const int4 d = P.desc[blockIdx.x];
  const int n = d.z, r = blockIdx.y * NG + threadIdx.x / LPG, c = threadIdx.x % LPG;
  if (n == 0 || r >= P.R) return;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, l = 0.f;
#pragma unroll 2
  for (int i = 0; i < n; ++i) {
    const float2 x = *reinterpret_cast<const float2 *>(P.ml + (piece(d.y, i) * P.R + r) * 2);
    const float4 v = *reinterpret_cast<const float4 *>(P.opart + (piece(d.y, i) * P.R + r) * D + 4 * c);
    const float top = fmaxf(m, x.x);
    const float f = m == -INFINITY ? 0.f : ex2_approx(m - top), w = x.x == -INFINITY ? 0.f : ex2_approx(x.x - top);
    m = top;
    l = f * l + w * x.y;
    a.x = f * a.x + w * v.x;
    a.y = f * a.y + w * v.y;
    a.z = f * a.z + w * v.z;
    a.w = f * a.w + w * v.w;
  }
  store_row(P, d.x, r, 4 * c, a, l);
}

// 5-D map of a cache: (column, slot, 128-byte group, head, page), box 128
// bytes x 16 slots x all groups, 128-byte swizzle.
static bool make_map(CUtensorMap *map, void *base, const sv_paged_kv *c, int D, int Hkv) {
  auto fn = attn::encode_fn();
  if (!fn) return false;
  const int es = c->dtype == SV_E4M3 ? 1 : 2;
  const cuuint32_t cols = 128 / es, groups = (cuuint32_t)(D * es / 128);
  cuuint64_t dims[5] = {cols, (cuuint64_t)c->page_size, groups, (cuuint64_t)Hkv, (cuuint64_t)c->num_pages};
  cuuint64_t strides[4] = {(cuuint64_t)c->slot_stride * es, 128, (cuuint64_t)c->head_stride * es,
                           (cuuint64_t)c->page_stride * es};
  cuuint32_t box[5] = {cols, (cuuint32_t)CHUNK, groups, 1, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(map, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, base, dims,
            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool F8, int MT>
static cudaError_t launch_main(const CUtensorMap &mk, const CUtensorMap &mv, Params &P, int ctas,
                               cudaStream_t s) {
  using LY = Layout<D, F8, MT>;
  const size_t fixed = 1024 + LY::RING + ((size_t)P.B + 1) * 4;
  // A multiple of the warps that take turns (NCW / MT), so that a ring slot's
  // chunks all fall to the same warps: a warp that came to a slot's next chunk
  // while another's was still on its way would take the barrier's phase of two
  // rounds ago for its own (phases are told apart by parity alone).
  constexpr int TURNS = NCW / MT * LY::NCH;
  P.stages = imin(MAX_STAGES, (int)((SMEM_LIMIT - fixed) / LY::STAGE)) / TURNS * TURNS & ~1;
  return launch_early(paged_kernel<D, F8, MT>, dim3(ctas), dim3(THREADS), fixed + (size_t)P.stages * LY::STAGE, s,
                mk, mv, P);
}

template <int D, bool F8>
static cudaError_t launch_tiles(const CUtensorMap &mk, const CUtensorMap &mv, Params &P, int ctas,
                                cudaStream_t s) {
  if (P.R <= 16) return launch_main<D, F8, 1>(mk, mv, P, ctas, s);
  if (P.R <= 32) return launch_main<D, F8, 2>(mk, mv, P, ctas, s);
  if (P.R <= 64) return launch_main<D, F8, 4>(mk, mv, P, ctas, s);
  return launch_main<D, F8, 8>(mk, mv, P, ctas, s);
}

template <int D>
static cudaError_t launch_all(bool f8, const CUtensorMap &mk, const CUtensorMap &mv, Params &P, int ctas,
                              cudaStream_t s) {
  cudaError_t e = f8 ? launch_tiles<D, true>(mk, mv, P, ctas, s) : launch_tiles<D, false>(mk, mv, P, ctas, s);
  if (e != cudaSuccess) return e;
  const int ng = JOIN_THREADS / (D / 4);
  return P.by_head ? launch_early(join_few_kernel<D>, dim3(P.B * P.Hkv, P.R), dim3(JOIN_THREADS), 0, s, P)
                   : launch_early(join_many_kernel<D>, dim3(ctas, (P.R + ng - 1) / ng), dim3(JOIN_THREADS), 0, s, P);
}

static size_t ws_bytes_for(int sms, int R, int D) {
  return (size_t)sms * (16 + 2 * (size_t)R * (D + 2) * sizeof(float));
}

}  // namespace paged
}  // namespace sv

using namespace sv;

extern "C" {

size_t paged_attn_workspace_bytes(int B, int M, int Hq, int Hkv, int D) {
  if (B < 1 || M < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return 0;
  if ((D != 128 && D != 256) || (long long)M * (Hq / Hkv) > paged::MAX_R) return 0;
  const int sms = imin(device_sm_count(), paged::MAX_CTAS);
  return sms <= 0 ? 0 : paged::ws_bytes_for(sms, M * (Hq / Hkv), D);
}

sv_status paged_kv_maps(const sv_paged_kv *cache, int Hkv, int D, void *maps_out, size_t maps_bytes) {
  static_assert(2 * sizeof(CUtensorMap) == SV_PAGED_MAPS_BYTES, "maps");
  if (Hkv < 1 || D < 1 || !maps_out || maps_bytes < SV_PAGED_MAPS_BYTES || !paged::aligned(maps_out, 8))
    return SV_ERR_INVALID_ARG;
  if (D != 128 && D != 256) return SV_ERR_UNSUPPORTED;
  const sv_status cs = paged::check_cache(cache, D);
  if (cs != SV_OK) return cs;
  CUtensorMap m[2];
  if (!paged::make_map(&m[0], cache->k, cache, D, Hkv) || !paged::make_map(&m[1], cache->v, cache, D, Hkv))
    return SV_ERR_CUDA;
  memcpy(maps_out, m, sizeof m);
  return SV_OK;
}

sv_status paged_attn(const sv_rows *q, const sv_paged_kv *cache, const int32_t *block_table,
                     int64_t table_stride, int table_width, const int32_t *kv_lens, const sv_rows *o, int B,
                     int M, int Hq, int Hkv, int D, float scale, int window, int sinks, void *workspace,
                     size_t ws_bytes, sv_stream_t stream) {
  if (B < 0 || M < 1 || Hq < 1 || Hkv < 1 || D < 1 || Hq % Hkv != 0) return SV_ERR_INVALID_ARG;
  if (window < 0 || sinks < 0 || table_width < (B > 0 ? 1 : 0) || table_stride < 0) return SV_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !(scale < INFINITY)) return SV_ERR_INVALID_ARG;
  if (D != 128 && D != 256) return SV_ERR_UNSUPPORTED;
  const int G = Hq / Hkv;
  if ((long long)M * G > paged::MAX_R || B > paged::MAX_B) return SV_ERR_UNSUPPORTED;
  if ((long long)B * M > 0x7fffffffLL || (long long)B * Hkv > 0x7fffffffLL) return SV_ERR_UNSUPPORTED;
  if (!paged::good_rows(q, (long long)B * M) || !paged::good_rows(o, (long long)B * M)) return SV_ERR_INVALID_ARG;
  const sv_status cs = paged::check_cache(cache, D);
  if (cs != SV_OK) return cs;
  if (B > 0 && (!block_table || !kv_lens)) return SV_ERR_INVALID_ARG;
  if (!paged::aligned(block_table, 4) || !paged::aligned(kv_lens, 4)) return SV_ERR_INVALID_ARG;
  // the groups of eight of a sequence's rows are counted in 31 bits, with room for a step
  if ((long long)M * Hq * D > 1LL << 33) return SV_ERR_UNSUPPORTED;
  // positions are 32-bit (with room for a window), and so is the line of units
  const long long cap = (long long)table_width * cache->page_size;
  if (cap > 0x40000000LL || window > 0x40000000 || (cap / paged::CHUNK + paged::HEAD_COST) * imax(B, 1) > 0x7fffffffLL / Hkv)
    return SV_ERR_UNSUPPORTED;
  if (B == 0) return SV_OK;
  const int sms = imin(device_sm_count(), paged::MAX_CTAS);
  if (sms <= 0) return SV_ERR_CUDA;
  const int R = M * G;
  if (!workspace || ws_bytes < paged::ws_bytes_for(sms, R, D)) return SV_ERR_WORKSPACE;
  if (!paged::aligned(workspace, 16)) return SV_ERR_INVALID_ARG;
  CUtensorMap mk, mv;
  if (cache->maps) {
    memcpy(&mk, cache->maps, sizeof mk);
    memcpy(&mv, static_cast<const char *>(cache->maps) + sizeof mk, sizeof mv);
  } else if (!paged::make_map(&mk, cache->k, cache, D, Hkv) || !paged::make_map(&mv, cache->v, cache, D, Hkv)) {
    return SV_ERR_CUDA;
  }
  paged::Params P{};
  P.q = *q;
  P.o = *o;
  P.table = block_table;
  P.table_stride = table_stride;
  P.width = table_width;
  P.lens = kv_lens;
  P.ks = cache->k_scale;
  P.vs = cache->v_scale;
  P.desc = static_cast<int4 *>(workspace);
  P.opart = reinterpret_cast<float *>(P.desc + sms);
  P.ml = P.opart + (size_t)2 * sms * R * D;
  P.err = device_error_word();
  if (!P.err) return SV_ERR_CUDA;
  P.B = B;
  P.M = M;
  P.Hkv = Hkv;
  P.G = G;
  P.R = R;
  P.sl2e = scale * 1.4426950408889634f;
  P.window = window;
  P.sinks = sinks;
  P.page_size = cache->page_size;
  P.num_pages = (int)cache->num_pages;
  P.min_units = 8;
  P.by_head = (long long)B * Hkv <= sms ? 1 : 0;
  P.stall = launch_flags() & SV_LAUNCH_TEST_STALL_COPY ? 1 : 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool f8 = cache->dtype == SV_E4M3;
  return from_cuda(D == 256 ? paged::launch_all<256>(f8, mk, mv, P, sms, s)
                            : paged::launch_all<128>(f8, mk, mv, P, sms, s));
}

}  // extern "C"
