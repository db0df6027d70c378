// chunk_attn.cu -- attention of ragged chunks of new tokens over a paged cache
// that already holds them, with an optional sliding window and a few first
// tokens that stay visible.
//
// Row i of a sequence's nq new rows stands at position p = len - nq + i and sees
// position j iff j <= p and (no window, or j > p - window, or j < sinks):
//   O = softmax_j(scale <Q, K_j>) V,   zeros where nothing is seen.
//
// What bounds it: 4 * D * Hq operations per visible (row, position) pair, so the
// tensor cores; for few rows the stream of the cache.  The products, the softmax
// between them and the tiles are window_attn's (128 query rows of one KV head a tile,
// S and P in tensor memory, O accumulated there); what differs:
//  * Keys and values come from pages: a copy is R = 16, 32 or 64 slots (a divisor of the
//    page size), one lane of the copying warp a copy, each looking its page up a
//    block ahead.  Blocks of a window begin at a multiple of R.
//  * The work is a line of all items (tiles of all KV heads), each as long as its
//    blocks of 128 keys and HEAD_COST for what it costs beside them, and every CTA (one
//    per SM) takes an equal piece of it: a few rows behind a long cache load all SMs, and ragged
//    batches load them alike.  A cut near an item's end moves there.  The pieces of a cut item leave O
//    (fp32), maximum and sum in the workspace, and a second kernel joins them.
//  * Slots that no row of the sequence sees may hold anything: their scores are
//    masked, and their values are overwritten with zeros before the product.
//  * e4m3 pages: keys are operands as they land, against queries in two e4m3 parts behind a power of two
//    per row (what the first part leaves is the second: exact down to 2^-9 of a row's largest element, off
//    by 2^-17 of that below).  Values meet probabilities, which take more than e4m3 parts: their copies
//    land in the second halves of their slots, and four more warps spread them out to fp16 tiles there
//    (each value exactly).  Probabilities are taken 2^10 times as large, and their sum with them, so that
//    those down to 2^-24 of the maximum keep 2^-11 (smaller ones are off by 2^-35 of it; the
//    maximum that they refer to is raised when a block exceeds it by more than 2^5).
//
// Measured (GB300, whole calls; the products' time at 1893 TFLOP/s): 2048 rows behind 30000
// positions, 24 heads of 256 over 4, 1.05 ms at 2.07 GHz and 1.16 at the 1.67 GHz that power leaves it (0.83); 13
// chunks of 1 to 777 rows behind 5000, 32 heads of 128 over 8, 116-120 us (67); 2 x 4001 rows under a window of
// 1024 over e4m3 pages 155 us (71; over bf16 pages 129); 61 rows behind 16000 over e4m3 pages 38-42 us, of which 9
// pass before the first product and 5 behind the last.  A block of two tiles takes 2900 clocks, of which 2050 are
// products: each tile's chain of scores, softmax and second product; an item costs 6000 more, 9000 with queries
// to turn.
#include "paged.cuh"
#include "tcgen05.cuh"

namespace sv {
namespace attn {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // attn.cu
}
namespace chunk {

constexpr int ROWS = 128;           // rows of a tile (TMEM lanes)
constexpr int BN = 128;             // keys of a block
constexpr int MAX_B = 4096;
constexpr int HEAD_COST = 2;        // blocks' time that an item takes beside its blocks
// Shared memory: barriers, the CTA's cuts (256), more barriers (280), the item
// (400), halves' exchange (512), prefix sums (2560; after the ring if longer), then the query
// tiles and the ring.
constexpr int HEADER = 3 * 1024, PREFIX = 2560, CUTS = 256, INFO = 400;

// Two tiles a CTA (D = 128), or one with two S buffers and two threads a row.
template <int D, int TILES, bool F8>
struct Cfg {
  static constexpr int NT = TILES;
  static constexpr int NSB = TILES == 2 ? 1 : 2;  // S buffers per tile
  static constexpr int SOFT = 8;                  // softmax warps
  static constexpr int HALVES = TILES == 2 ? 1 : 2;  // threads that share a row
  // Ring slots: a whole K or V block at D = 128, at D = 256 half of its columns
  // (K) or of its keys (V).
  static constexpr int SLOT = 32768, RAW = SLOT / 2;  // (e4m3: where a copy of values lands)
  static constexpr int PARTS = BN * D * 2 / SLOT;  // slots of a K block (of a V block)
  // e4m3 keys are operands as they land: a slot a block
  static constexpr int KSLOT = F8 ? BN * D : SLOT, KPARTS = F8 ? 1 : PARTS;
  static constexpr int KG = D / 64 / PARTS;        // 64-column groups of a K slot (bf16)
  static constexpr int VK = BN / PARTS;            // keys of a V slot
  static constexpr int THREADS = (SOFT + (F8 ? 8 : 4)) * 32;
  static constexpr int QBYTES = ROWS * D * 2;
  static constexpr int RING = HEADER + NT * QBYTES;
  // slots of the K and the V ring: 160 KB, or 128 beside long prefix sums and with e4m3 pages
  // (At D = 256 a block takes two slots of each, and the next block's keys are needed first.)
  static constexpr int NK = F8 ? 2 : D == 256 ? 3 : 2, NV = F8 ? (D == 256 ? 2 : 3) : 5 - NK;
  static constexpr int LESS_K = 2, LESS_V = F8 ? NV : 2;
  static_assert(NK * KSLOT + NV * SLOT == (F8 ? 128 : 160) * 1024 && LESS_K * KSLOT + LESS_V * SLOT == 128 * 1024, "ring");
  static constexpr int BEHIND = RING + 128 * 1024;  // prefix sums
  // tensor memory: O per tile, then the S buffers (P over S)
  static constexpr uint32_t TO = 0, TS = NT * D;
  static_assert(NT * D + NT * NSB * BN <= 512, "tensor memory");
  // registers: as many as the threads start with
  static constexpr int SOFT_REGS = F8 ? (NT == 2 ? 216 : 184) : 216, OTHER_REGS = F8 && NT == 2 ? 40 : 72;
  static_assert(256 * SOFT_REGS + (THREADS - 256) * OTHER_REGS <= (65536 / THREADS / 8 * 8) * THREADS, "registers");
  // log2 of the factor on probabilities and their sum, and of the largest P against an
  // old maximum, factor included
  static constexpr float LIFT = F8 ? 10.f : 0.f, RESCALE = F8 ? 5.f : 8.f;
};

// Item that a CTA begins and does not end: its pieces are this CTA's second and the first of
// each of the pieces - 1 CTAs behind it (0: none).
struct Cut {
  int h, q0, rows, pieces;
};

struct Params {
  sv_rows o;
  const int *cu_q, *lens, *table;
  long long table_stride;
  int width, page_size, num_pages;
  int R, piece;  // slots of a copy; first keys that may share a block with others (whole copies)
  const float *ks, *vs;
  float *opart;  // [2 * ctas][NT][D / 4][ROWS][4] unnormalised O
  float2 *ml;    // [2 * ctas][NT * ROWS] maximum (log2 domain) and sum
  Cut *cuts;     // [ctas]
  unsigned *err;
  int B, Tq, Hkv, G, PT;  // PT: positions per tile
  int most;          // tiles that sequences without common rows can have
  float sl2e;
  int window, sinks;
  int few_slots;  // long prefix sums take the place of some
  int stall;      // test aid: the first slot of the K ring never fills
};
constexpr int MAX_KEPT = 31;  // sequences whose offsets and lengths are kept in shared memory (int4 each)

struct Item {
  int b, h, q0;      // sequence, KV head, first row
  int rows;          // positions of the item
  int p0, len;       // position of its first row; slots of the sequence
  int from;          // positions before it that are not among the first `sinks` are seen by no row of the sequence
  // Blocks: ns over the first keys, then those from key w0 on; n in all.  Up to
  // `piece` first keys far from the window (ns = 0, w0 > 0, sinks) need no block:
  // keys 0..piece-1 stand in the first block's first rows, for w0..w0+piece-1.
  int ns, skip, n;
  __device__ __forceinline__ int base(int j) const { return j * BN + (j < ns ? 0 : skip); }
};
// The part of an item that is this CTA's: blocks j0..j1-1.
struct Part {
  int id, j0, j1;
};

// Rows of sequence b, 0 if its offsets are out of order or out of range.
__device__ __forceinline__ int rows_of(const Params &P, int b, bool report) {
  const int q0 = P.cu_q[b], q1 = P.cu_q[b + 1];
  if (q0 < 0 || q1 < q0 || q1 > P.Tq) {
    if (report) atomicOr(P.err, ERR_INDEX);
    return 0;
  }
  return q1 - q0;
}
__device__ __forceinline__ int length_of(const Params &P, int b, bool report) {
  const long long cap = (long long)P.width * P.page_size;
  const int l = P.lens[b];
  if (l < 0 || l > cap) {
    if (report) atomicOr(P.err, ERR_INDEX);
    return l < 0 ? 0 : (int)cap;
  }
  return l;
}

// Tile `c` of the line (pre: tiles before a sequence, or, of few sequences, those, the first
// row, the rows and the length), for KV head h.
template <int NT>
__device__ __forceinline__ Item tile_at(const Params &P, const int *pre, int c, int h) {
  const bool kept = P.B <= MAX_KEPT;
  const int each = kept ? 4 : 1;
  int lo = 0, hi = P.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid * each] <= c) lo = mid; else hi = mid - 1;
  }
  const int b = lo, span = P.PT * NT;
  Item it;
  it.b = b;
  it.h = h;
  // a sequence's last tiles first: they see the most
  const int row0 = (pre[(b + 1) * each] - 1 - c) * span;
  int q0, nq;
  if (kept) {
    const int4 x = reinterpret_cast<const int4 *>(pre)[b];
    q0 = x.y, nq = x.z, it.len = x.w;
  } else {
    q0 = P.cu_q[b], nq = P.cu_q[b + 1] - q0, it.len = length_of(P, b, false);
  }
  it.q0 = q0 + row0;
  it.rows = imin(span, nq - row0);
  it.p0 = it.len - nq + row0;
  it.from = P.window > 0 ? imax(0, it.len - nq - P.window + 1) : 0;
  const int end = imax(0, it.p0 + it.rows);  // of the keys that some row sees
  const int start = P.window > 0 ? imin(end, imax(0, it.p0 - P.window + 1)) : 0;
  const int first = imin(P.sinks, end);
  it.ns = first > P.piece ? (first + BN - 1) / BN : 0;
  int w0 = first > P.piece || first == 0 ? start : imax(0, start - P.piece);
  w0 &= -P.R;
  if (w0 <= it.ns * BN) w0 = it.ns = 0;
  it.skip = w0 - it.ns * BN;
  it.n = it.ns + (end - w0 + BN - 1) / BN;
  return it;
}
template <int NT>
__device__ __forceinline__ Item item_at(const Params &P, const int *pre, int id) {
  const int c = id / P.Hkv;
  return tile_at<NT>(P, pre, c, id - c * P.Hkv);
}

// Whether the first keys stand in this block's first rows.
__device__ __forceinline__ bool heads(const Params &P, const Item &it, int j) {
  return j == 0 && it.ns == 0 && it.skip > 0 && P.sinks > 0;
}
// Position of row r of block j.
__device__ __forceinline__ int position(const Params &P, const Item &it, int j, int r) {
  return r < P.piece && heads(P, it, j) ? r : it.base(j) + r;
}
// Rows of block j that no row of the sequence sees (or none of the item): a..b-1, and those from c on.
struct Blind {
  int a, b, c;
  __device__ __forceinline__ bool operator()(int r) const { return (r >= a && r < b) || r >= c; }
};
__device__ __forceinline__ Blind blind(const Params &P, const Item &it, int j) {
  const int base = it.base(j);
  const bool h = heads(P, it, j);
  return Blind{h ? P.sinks : imax(0, P.sinks - base), h ? imax(P.piece, it.from - base) : it.from - base, it.len - base};
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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

__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t v) {  // to the nearest, in the low 16 bits
  uint32_t d;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f16x2 t, %1;\n\tmov.b32 %0, {t, 0};\n\t}\n" : "=r"(d) : "r"(v));
  return d;
}

__device__ __forceinline__ void tma_load_4d(void *smem_dst, const CUtensorMap *map, int c0, int c1, int c2,
                                            int c3, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(smem_dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void page_load(void *smem_dst, const CUtensorMap *map, int slot, int group, int head, int page,
                                          uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(smem_dst)),
      "l"(map), "r"(0), "r"(slot), "r"(group), "r"(head), "r"(page), "r"(smem_u32(bar))
      : "memory");
}

template <int D, int TILES, bool F8>
__global__ void __launch_bounds__(Cfg<D, TILES, F8>::THREADS, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                      const __grid_constant__ CUtensorMap mapV, const __grid_constant__ Params P) {
  using C = Cfg<D, TILES, F8>;
  constexpr int NT = C::NT, NSB = C::NSB, PARTS = C::PARTS, VK = C::VK, KG = C::KG, SLOT = C::SLOT, KSLOT = C::KSLOT;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw;
  // The swizzled tiles need 1024-byte alignment, which the first dynamic byte
  // has in a kernel without static shared memory.
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicOr(P.err, ERR_TIMEOUT);
    return;
  }
  uint64_t *full = reinterpret_cast<uint64_t *>(smem);  // [2][5] slots of the K ring, of the V ring
  uint64_t *empty = full + 10;     // [2][5]
  uint64_t *s_full = empty + 10;   // [2] per S buffer
  uint64_t *p_full = s_full + 2;   // [2] per S buffer: P written over it
  uint64_t *o_done = p_full + 2;   // [2] per S buffer: the second product of its P done
  uint64_t *o_free = o_done + 2;   // [2] O read out
  uint64_t *q_full = o_free + 2;   // [2] queries of a tile of the item landed
  uint64_t *q_free = q_full + 2;   // last S product of the item done
  // (31 barriers, 248 bytes; the rest stands behind the cuts)
  uint64_t *more = reinterpret_cast<uint64_t *>(smem + 280);
  uint64_t *idle = more, *p_half = more + 1;  // p_half [2] one S buffer: P of the first half of a block's keys written
  uint64_t *q_ready = more + 3, *copied = more + 5;  // e4m3: [2] queries of a tile turned, [5] copies of values landed
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + CUTS + 16);
  int2 *cut = reinterpret_cast<int2 *>(smem + CUTS);  // [2] item and block where this CTA begins, and the next one
  Item *info_it = reinterpret_cast<Item *>(smem + INFO);  // of the item whose queries landed
  int *info = reinterpret_cast<int *>(smem + INFO + 48);  // its first block, its end, its tiles
  float *xchg = reinterpret_cast<float *>(smem + 512);  // [2][2 halves][ROWS] maxima, then sums
  uint8_t *qs = smem + HEADER;
  uint8_t *ring = smem + C::RING;
  const int NK = P.few_slots ? C::LESS_K : C::NK, NV = P.few_slots ? C::LESS_V : C::NV;
  int *pre = reinterpret_cast<int *>(smem + (P.few_slots ? C::BEHIND : PREFIX));

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 0) {  // a barrier a lane, in the order above
    if (lane < 31) {
      const int of_values = F8 && lane >= 5 && lane < 10 ? 4 : 1, softmax = 4 * C::HALVES;
      const int n = lane < 10 ? of_values + (lane == 0 ? P.stall : 0)
                              : (lane == 22 || lane == 23 || lane == 26 || lane == 27) ? softmax : 1;
      mbar_init(&full[lane], n);
    }
    if (lane < 10) mbar_init(&more[lane], lane == 1 || lane == 2 ? 4 : lane == 3 || lane == 4 ? 4 * C::HALVES : 1);
    fence_barrier_init();
  }
  if (warp == C::SOFT) {
    tc::tmem_alloc(tmem_slot, 512u);
    tc::tmem_relinquish();
  }
  // rows of the query tiles that no load writes stay zero
  const int used = P.PT * P.G;
  for (int x = tid; x < NT * (ROWS - used) * (D / 8); x += C::THREADS) {
    const int t = x / ((ROWS - used) * (D / 8)), y = x % ((ROWS - used) * (D / 8));
    const int r = used + y / (D / 8), c = y % (D / 8);
    *reinterpret_cast<uint4 *>(qs + t * C::QBYTES + (c >> 3) * ROWS * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  // Values of slots that are not copied meet probabilities of zero and have to be finite.
  for (int x = tid; x < NV * SLOT / 16; x += C::THREADS)
    reinterpret_cast<uint4 *>(ring + NK * KSLOT)[x] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async();
  pdl_wait();

  // ---- prefix sums of the sequences' tiles ----
  // Offsets that fall and rise again can name the same rows thousands of times:
  // the sums stay at the top instead of wrapping, and then no item is left.
  auto sum = [](int a, int b) { return (int)min((unsigned)a + (unsigned)b, 0x7fffffffu); };
  // inclusive sums over the block, and the total
  auto scan = [&](int x, int &all) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x = sum(x, y);
    }
    if (lane == 31) xchg[warp] = __int_as_float(x);
    __syncthreads();
    int before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < C::THREADS / 32; ++w) {
      const int y = __float_as_int(xchg[w]);
      if (w < warp) before = sum(before, y);
      all = sum(all, y);
    }
    __syncthreads();
    return sum(before, x);
  };
  const bool report = blockIdx.x == 0;
  int tiles = 0;
  if (P.B <= MAX_KEPT) {  // a sequence a lane, in every warp
    const int q0 = lane < P.B ? P.cu_q[lane] : 0, nq = lane < P.B ? rows_of(P, lane, report) : 0;
    const int len = lane < P.B ? length_of(P, lane, report) : 0, nt = (nq + P.PT * NT - 1) / (P.PT * NT);
    int x = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x = sum(x, y);
    }
    if (warp == 0 && lane < P.B) reinterpret_cast<int4 *>(pre)[lane] = make_int4(x - nt, q0, nq, len);
    tiles = __shfl_sync(0xffffffffu, x, 31);
  } else {
    for (int b0 = 0; b0 < P.B; b0 += C::THREADS) {
      const int b = b0 + tid;
      const int nq = b < P.B ? rows_of(P, b, report) : 0;
      if (b < P.B) length_of(P, b, report);
      const int nt = (nq + P.PT * NT - 1) / (P.PT * NT);
      int all;
      const int x = scan(nt, all);
      if (b < P.B) pre[b] = sum(tiles, x) - nt;
      tiles = sum(tiles, all);
    }
  }
  if (tiles > P.most) {
    if (tid == 0 && blockIdx.x == 0) atomicOr(P.err, ERR_INDEX);
    tiles = 0;
  }
  if (tid == 0) pre[P.B <= MAX_KEPT ? 4 * P.B : P.B] = tiles;
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = *tmem_slot;

  // ---- this CTA's piece of the line ----
  {
    auto weight = [&](int c) { return c < tiles ? tile_at<NT>(P, pre, c, 0).n + HEAD_COST : 0; };
    int per_head = 0, all = 0, mine = 0, upto = 0;
    for (int c0 = 0; c0 < tiles; c0 += C::THREADS) {
      mine = weight(c0 + tid);
      upto = scan(mine, all);
      per_head += all;  // (in 31 bits with the heads: checked on the host)
    }
    // (no CTA takes less than four blocks' time, so that no two cuts coincide)
    const int W = per_head * P.Hkv, ctas = imin(gridDim.x, imax(1, W / 4));
    const int share = W / ctas, rest = W - share * ctas;
    auto line = [&](int x) { return x = imin(x, ctas), share * x + rest * x / ctas; };  // W * x / ctas
    const int at[2] = {line(blockIdx.x), line(blockIdx.x + 1)};
    // A cut this near to an item's beginning or end moves there: what cutting costs (both
    // pieces' O through the workspace) is a block or two.
    const int near = imax(3, share / 16);
    if (tid < 2) cut[tid] = make_int2(tiles * P.Hkv, 0);
    if (tid == 0) P.cuts[blockIdx.x].pieces = 0;
    __syncthreads();
    int before = 0;
    for (int c0 = 0; c0 < tiles; c0 += C::THREADS) {
      const bool again = tiles > C::THREADS;
      const int c = c0 + tid, w = again ? weight(c) : mine;
      const int x = before + (again ? scan(w, all) : upto) - w;  // tiles' weight before this one
      before += all;
#pragma unroll 1
      for (int e = 0; e < 2; ++e) {
        const int y = at[e] - x * P.Hkv;
        if (y < 0 || y >= w * P.Hkv) continue;
        const int h = y / w, j = y - h * w - HEAD_COST, n = w - HEAD_COST, id = c * P.Hkv + h;
        cut[e] = j < near ? make_int2(id, 0) : n - j < near ? make_int2(id + 1, 0) : make_int2(id, j);
        if (e == 1 && j >= near && n - j >= near && at[0] - HEAD_COST - near < at[1] - j - HEAD_COST) {
          // cut at its end, and not in the same item at its beginning: the item begins here; every
          // CTA up to the last cut in it has a piece
          const int last_cut = at[1] - j + n - near;  // of the line, the last place to cut it
          const int last = (int)lmin(ctas - 1, (((long long)last_cut + 1) * ctas - 1) / W);  // the last x with line(x) <= last_cut
          const Item it = tile_at<NT>(P, pre, c, h);
          P.cuts[blockIdx.x] = Cut{it.h, it.q0, it.rows, 1 + imax(1, last - (int)blockIdx.x)};
        }
      }
    }
    __syncthreads();
  }
  const int parts = cut[1].x - cut[0].x + (cut[1].y > 0 ? 1 : 0);
  // this CTA's k-th part (its cuts out of shared memory each time: no role has a register to spare)
  const uint32_t cut_at = smem_u32(cut);
  auto id_of = [&](int k) { return (int)lds64(cut_at).x + k; };
  auto part_of = [&](int k, const Item &it) {
    const uint2 a = lds64(cut_at), z = lds64(cut_at + 8);
    return Part{(int)a.x + k, k == 0 ? (int)a.y : 0, (int)a.x + k == (int)z.x ? (int)z.y : it.n};
  };

  if (warp >= C::SOFT) {
    setmaxnreg_dec<C::OTHER_REGS>();
    if (warp == C::SOFT + 1 || warp == C::SOFT + 3) {
      // -------------------- copies: K blocks by one warp, V blocks by the other --
      const bool is_v = warp == C::SOFT + 3;
      uint64_t *landed = is_v ? (F8 ? copied : full + 5) : full, *free = empty + (is_v ? 5 : 0);
      uint8_t *slots = ring + (is_v ? NK * KSLOT : 0);
      const int NS = is_v ? NV : NK, size = is_v ? SLOT : KSLOT, per_block = is_v ? PARTS : C::KPARTS;
      // A lane a piece of R rows (of a column group), all pieces of a slot at once.
      int first, gap, group, place;  // its first row in slot 0 of a block, from slot to slot, column group, where in the slot
      int step = 0;                  // of the column group from slot to slot
      if (F8) {
        constexpr int groups = D / 128;  // of 128 columns
        const int p = lane / groups;
        first = p * P.R, gap = is_v ? VK : 0, group = lane % groups;
        place = (is_v ? C::RAW : 0) + group * (is_v ? VK : BN) * 128 + p * P.R * 128;
      } else if (is_v) {
        first = lane * P.R, gap = VK, group = 0, place = lane * P.R * 128 * (D / 64);
      } else {
        first = lane / KG * P.R, gap = 0, group = lane % KG, step = KG, place = ((lane % KG) * BN + first) * 128;
      }
      const bool here = first < (is_v ? VK : BN);
      const uint32_t bytes = (uint32_t)P.R * 128 * (!F8 && is_v ? D / 64 : 1);
      // A piece's page and its slot there: page -1 where no row sees any slot of it, past the cache
      // where its entry is (which reads as zeros).  Values behind the sequence's end are read as the page
      // behind the last, as zeros: their place holds what another item left, which may be anything.
      struct Place {
        int page, slot;
      };
      auto look = [&](const Item &it, int j, int x) {
        const int pos = position(P, it, j, first + x * gap);
        if (!F8 && is_v && here && pos >= it.len) return Place{P.num_pages, 0};
        if (!here || pos >= it.len || (pos >= P.sinks && pos + P.R <= it.from)) return Place{-1, 0};
        const int e = pos / P.page_size;
        const int page = P.table[it.b * P.table_stride + e];
        return Place{page == P.num_pages ? -2 : page, page == -1 ? ~(pos - e * P.page_size) : pos - e * P.page_size};
      };
      bool ok = true;
      uint32_t q = 0, parity = 1;
      int slot = 0;
      Item it{};
      Part pt{0, 0, 0};
      int k = -1;
      auto next_part = [&]() {  // the next one with blocks
        do {
          if (++k >= parts) return false;
          it = item_at<NT>(P, pre, id_of(k));
          pt = part_of(k, it);
        } while (pt.j0 == pt.j1);
        return true;
      };
      bool more_parts = next_part();
      int j = pt.j0, x = 0, h = it.h;
      Place at = more_parts ? look(it, j, x) : Place{-1, 0};
      while (more_parts) {
        // the one after it is looked up before this one's slot is waited for
        const int now_x = x;
        h = it.h;
        if (++x == per_block) x = 0, ++j;
        if (j == pt.j1) {
          more_parts = next_part();
          j = pt.j0;
        }
        const Place next = more_parts ? look(it, j, x) : Place{-1, 0};
        if (ok && lane == 0) ok = mbar_wait(&free[slot], parity, P.err);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        bool live = at.page != -1;
        // (an entry of -1 that is needed counts as a page past the cache: told apart by the slot)
        if (at.slot < 0) live = true, at.slot = ~at.slot;
        const uint32_t n = __popc(__ballot_sync(0xffffffffu, live));
        if (lane == 0) mbar_arrive_expect_tx(&landed[slot], n * bytes);
        __syncwarp();
        if (live) {
          if (at.page < 0 || at.page > P.num_pages) {
            atomicOr(P.err, ERR_INDEX);
            at.page = P.num_pages;
          }
          page_load(slots + slot * size + place, is_v ? &mapV : &mapK, at.slot, group + now_x * step, h, at.page, &landed[slot]);
        }
        at = next;
        ++q;
        if (++slot == NS) {
          slot = 0;
          parity ^= 1;
        }
      }
      if (!ok && lane == 0) {  // no copy may outlive the CTA
        const uint32_t first = q > (uint32_t)NS ? q - NS : 0u;
        for (uint32_t qq = first; qq < q && mbar_wait(&landed[qq % NS], (qq / NS) & 1, P.err); ++qq) {
        }
      }
      __syncwarp();
    } else if (warp == C::SOFT + 2) {
      // --------------------------------------------------- queries --
      if (lane == 0) {
        bool ok = true;
        uint32_t c = 0, c1 = 0;  // parts with work so far, those with a second tile
        for (int k = 0; k < parts && ok; ++k) {
          const Item it = item_at<NT>(P, pre, id_of(k));
          const Part pt = part_of(k, it);
          if (pt.j0 == pt.j1) continue;
          if (c > 0) ok = mbar_wait(q_free, (c - 1) & 1, P.err);
          if (!ok) break;
          ++c;
          const int nt = it.rows > P.PT ? NT : 1;
          c1 += nt - 1;
          *info_it = it;
          info[0] = pt.j0, info[1] = pt.j1, info[2] = nt;
          for (int t = 0; t < nt; ++t) {
            mbar_arrive_expect_tx(&q_full[t], (uint32_t)(used * D * 2));
#pragma unroll
            for (int g = 0; g < D / 64; ++g)
              tma_load_4d(qs + t * C::QBYTES + g * ROWS * 128, &mapQ, 0, it.h * P.G, it.q0 + t * P.PT, g, &q_full[t]);
          }
        }
        if (ok && c > 0) ok = mbar_wait(q_free, (c - 1) & 1, P.err);
        if (ok) {  // no part is left
          info[0] = info[1] = 0;
          mbar_arrive(q_full);
        } else {
          if (c > 0) mbar_wait(q_full, (c - 1) & 1, P.err);
          if (c1 > 0) mbar_wait(q_full + 1, (c1 - 1) & 1, P.err);
        }
      }
      __syncwarp();
    } else if (F8 && warp >= C::SOFT + 4) {
      // ------------------------------------------------ e4m3 values to fp16 --
      const int i = tid - (C::SOFT + 4) * 32;
      bool ok = true;
      int at_slot = 0;
      uint32_t phase = 0;
      // One slot: its copy stands in the second half.  The half of the columns whose fp16 tiles lie in the
      // first half comes first, then, once all have read them, the rest.
      auto turn = [&](const Item &it, int j, int x) {
        constexpr bool whole = VK == 64;             // a half of the copy: all pieces of 64 rows, or half of those of 128
        constexpr int gap = whole ? 16 : 32;         // rows between a thread's pieces
        if (ok) ok = spin_wait(&copied[at_slot], phase, P.err);
        ok = __all_sync(0xffffffffu, ok);
        uint8_t *base = ring + NK * KSLOT + at_slot * SLOT;
        const int r0 = whole ? i >> 3 : i >> 2, c = whole ? i & 7 : i & 3;
        Blind none{0, 0, BN};
        if (j <= it.ns || j + 1 == it.n) none = blind(P, it, j);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint8_t *raw = base + C::RAW + (whole ? half * 8192 + r0 * 128 + c * 16 : r0 * 128 + (4 * half + c) * 16);
          uint4 w[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) w[y] = *reinterpret_cast<const uint4 *>(raw + y * gap * 128);
          if (none.a < none.b || none.c < BN) {  // slots that no row sees count as zeros
#pragma unroll
            for (int y = 0; y < 4; ++y)
              if (none(x * VK + r0 + gap * y)) w[y] = make_uint4(0u, 0u, 0u, 0u);
          }
          if (half == 1) named_barrier(6, 128);
          uint8_t *out = base + half * C::RAW + (whole ? (c >> 2) * 8192 : 0) + r0 * 128;
          const uint32_t a0 = ((2 * (c & 3)) ^ (r0 & 7)) << 4, a1 = ((2 * (c & 3) + 1) ^ (r0 & 7)) << 4;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            *reinterpret_cast<uint4 *>(out + y * gap * 128 + a0) =
                make_uint4(e4m3x2_to_f16x2(w[y].x), e4m3x2_to_f16x2_hi(w[y].x), e4m3x2_to_f16x2(w[y].y), e4m3x2_to_f16x2_hi(w[y].y));
            *reinterpret_cast<uint4 *>(out + y * gap * 128 + a1) =
                make_uint4(e4m3x2_to_f16x2(w[y].z), e4m3x2_to_f16x2_hi(w[y].z), e4m3x2_to_f16x2(w[y].w), e4m3x2_to_f16x2_hi(w[y].w));
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[5 + at_slot]);
        if (++at_slot == NV) at_slot = 0, phase ^= 1;
      };
      for (int k = 0; k < parts; ++k) {
        const Item it = item_at<NT>(P, pre, id_of(k));
        const Part pt = part_of(k, it);
        if (pt.j0 == pt.j1) continue;
        for (int j = pt.j0; j < pt.j1; ++j)
#pragma unroll 1
          for (int x = 0; x < PARTS; ++x) turn(it, j, x);
      }
      __syncwarp();
    } else if (warp == C::SOFT) {
      // ------------------------------------------------- MMA issuer --
      constexpr uint32_t IDS = F8 ? tc::idesc_e4m3_f32(ROWS, BN) : tc::idesc_bf16_f32(ROWS, BN, false);
      constexpr uint32_t IDO = F8 ? tc::idesc_f16_f32(ROWS, D, true) : tc::idesc_bf16_f32(ROWS, D, true);
      // rows of a piece of values: a copy's (bf16), or all of a slot
      const int VR = F8 ? VK : P.R;
      // descriptors: queries and keys K-major, values with rows along K
      const uint64_t dq = tc::smem_desc_sw128(smem_u32(qs), 16, 1024), dk = tc::smem_desc_sw128(smem_u32(ring), 16, 1024);
      const uint64_t dv = tc::smem_desc_sw128(smem_u32(ring + NK * KSLOT), VR * 128, 1024);
      const uint32_t q_lo = (uint32_t)dq, q_hi = (uint32_t)(dq >> 32), k_lo = (uint32_t)dk, k_hi = (uint32_t)(dk >> 32);
      const uint32_t v_lo = (uint32_t)dv, v_hi = (uint32_t)(dv >> 32);
      // of 16 keys' step ks in a slot of values: piece by piece, all column groups of one together
      const int lg = F8 ? 4 : P.R == 64 ? 2 : P.R == 32 ? 1 : 0, steps = (1 << lg) - 1;  // log2 of steps a piece
      const uint32_t piece = (uint32_t)VR * 128 * (D / 64) / 16;
      const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
      const bool leader = tc::elect_one();
      // After a wait that ran out the warp goes through the rest of the part
      // without waiting or issuing, so that its lanes stay together.
      bool ok = true;
      auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (ok) ok = spin_wait(bar, parity, P.err);
      };
      struct Cursor {  // a ring's next slot
        int slot;
        uint32_t parity;
        __device__ __forceinline__ void step(int slots) {
          if (++slot == slots) {
            slot = 0;
            parity ^= 1;
          }
        }
      };
      Cursor ck{0, 0}, cv{0, 0};
      uint32_t c = 0;                     // parts with work so far
      uint32_t sj[NT] = {}, pj[NT] = {};  // blocks of each tile: S issued, P consumed
      uint32_t oc[NT] = {};               // parts of each tile
      while (ok) {
        wait(q_full, c & 1);
        // (a limit may run out in some lanes while the phase completes for others)
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++c;
        const int j0 = __shfl_sync(0xffffffffu, info[0], 0), j1 = __shfl_sync(0xffffffffu, info[1], 0);
        const int nt = __shfl_sync(0xffffffffu, info[2], 0);
        if (j1 == 0) break;
        const Item it = *info_it;  // (the next part's may stand there before this one's last product)
        if (!F8 && nt == 2) wait(q_full + 1, oc[NT - 1] & 1);
        // S of the next block for tiles ta..tb1-1; `release`: they are its last
        auto issue_s = [&](int ta, int tb1, bool release, bool last) {
          Cursor at = ck;
#pragma unroll
          for (int x = 0; x < C::KPARTS; ++x) {
            if (ta == 0) wait(&full[at.slot], at.parity);  // (tile 1 follows tile 0)
            tc::fence_after_sync();
            if (leader && ok) {
              const uint32_t ka = k_lo + at.slot * (KSLOT / 16);
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                if (t < ta || t >= tb1) continue;
                const uint32_t sb = NSB == 2 ? (sj[0] & 1) : (uint32_t)t;
                if constexpr (F8) {  // 32 columns a step, both parts of the queries
#pragma unroll
                  for (int ks = 0; ks < D / 16; ++ks)
                    tc::mma_e4m3(tb + C::TS + sb * BN, q_lo + (t * C::QBYTES + (ks >> 2) * ROWS * 128 + (ks & 3) * 32) / 16, q_hi,
                                 ka + ((ks >> 3) * BN * 128 + ((ks >> 1) & 3) * 32) / 16, k_hi, IDS, ks > 0 ? 1u : 0u);
                } else {
#pragma unroll
                  for (int ks = 0; ks < KG * 4; ++ks)
                    tc::mma_bf16(tb + C::TS + sb * BN,
                                 q_lo + (t * C::QBYTES + (x * KG + (ks >> 2)) * ROWS * 128 + (ks & 3) * 32) / 16, q_hi,
                                 ka + ((ks >> 2) * BN * 128 + (ks & 3) * 32) / 16, k_hi, IDS,
                                 (x > 0 || ks > 0) ? 1u : 0u);
                }
                if (x == C::KPARTS - 1) tc::commit(&s_full[sb]);
              }
              if (release) tc::commit(&empty[at.slot]);
              if (last && x == C::KPARTS - 1) tc::commit(q_free);
            }
            at.step(NK);
          }
          if (release) ck = at;
#pragma unroll
          for (int t = 0; t < NT; ++t)
            if (t >= ta && t < tb1) ++sj[t];
        };
        if (F8) {  // a tile as soon as its queries are turned
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if (t >= nt) continue;
            wait(q_ready + t, oc[t] & 1);
            issue_s(t, t + 1, t == nt - 1, t == nt - 1 && j1 - j0 == 1);
          }
        } else {
          issue_s(0, nt, true, j1 - j0 == 1);
        }
        for (int j = j0; j < j1; ++j) {
          const bool more = j + 1 < j1;
          if (NSB == 2 && more) issue_s(0, 1, true, j + 2 == j1);  // runs during this block's softmax
          // blocks with slots that no row sees: those up to a window's first, and the last
          const bool some = !F8 && (j <= it.ns || j + 1 == it.n);  // (e4m3: zeros already)
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if (t >= nt) continue;
            const uint32_t sb = NSB == 2 ? (pj[t] & 1) : (uint32_t)t;
            if (j == j0 && oc[t] > 0) wait(&o_free[t], (oc[t] - 1) & 1);
            if (NSB == 2) wait(&p_full[sb], (pj[t] >> 1) & 1);
            Cursor at = cv;
#pragma unroll
            for (int x = 0; x < PARTS; ++x) {
              if (t == 0) wait(&full[5 + at.slot], at.parity);
              if (some && t == 0) {
                const Blind none = blind(P, it, j);
                const int upto = (none.c + P.R - 1) & -P.R;  // (pieces behind are zeros)
                uint8_t *vb = ring + NK * KSLOT + at.slot * SLOT;
                auto clear = [&](int r0, int r1) {  // rows of the block, those of this slot
                  r0 = imax(r0 - x * VK, 0), r1 = imin(r1 - x * VK, VK);
                  for (int e = lane; e < (r1 - r0) * (D / 8); e += 32) {
                    const int r = r0 + e / (D / 8), y = e % (D / 8);
                    *reinterpret_cast<uint4 *>(vb + (r / P.R) * P.R * 128 * (D / 64) + (y >> 3) * P.R * 128 + (r % P.R) * 128 + (y & 7) * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
                  }
                };
                clear(none.a, imin(none.b, BN));
                clear(none.c, imin(upto, BN));
                fence_proxy_async();
                __syncwarp();
              }
              // one S buffer: the first half of the keys while the second's P is made
              constexpr int STEPS = NSB == 1 ? 2 : 1;
#pragma unroll
              for (int y = 0; y < STEPS; ++y) {
                if (NSB == 1) wait(y == 0 ? &p_half[sb] : &p_full[sb], pj[t] & 1);
                tc::fence_after_sync();
                if (leader && ok) {
                  const uint32_t va = v_lo + at.slot * (SLOT / 16);
#pragma unroll
                  for (int ks = y * (VK / 16 / STEPS); ks < (y + 1) * (VK / 16 / STEPS); ++ks) {
                    const uint32_t vo = (uint32_t)(ks >> lg) * piece + (uint32_t)(ks & steps) * (2048 / 16);
                    tc::mma_bf16_ts(tb + C::TO + t * D, tb + C::TS + sb * BN + (x * (VK / 16) + ks) * 8,
                                    va + vo, v_hi, IDO, (x > 0 || ks > 0) ? 1u : (uint32_t)(j > j0));
                  }
                }
              }
              if (leader && ok) {
                if (x == PARTS - 1) tc::commit(&o_done[sb]);
                if (t == nt - 1) tc::commit(&empty[5 + at.slot]);
              }
              at.step(NV);
            }
            if (t == nt - 1) cv = at;
            ++pj[t];
            if (NSB == 1 && more) issue_s(t, t + 1, t == nt - 1, t == nt - 1 && j + 2 == j1);
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
          if (t < nt) ++oc[t];
        ok = __all_sync(0xffffffffu, ok);
      }
      if (leader) {  // every product issued above has completed before TMEM is released
        tc::commit(idle);
        spin_wait(idle, 0, P.err);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------ softmax --
    setmaxnreg_inc<C::SOFT_REGS>();
    constexpr int HALVES = C::HALVES, COLS = BN / HALVES;  // keys of a block that are this thread's
    const int t = HALVES == 1 ? warp >> 2 : 0;  // tile
    const int hf = HALVES == 1 ? 0 : warp >> 2;  // half of a block's keys, and of O's columns
    const int r = (warp & 3) * 32 + lane;       // row = TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const int ir = r / P.G;                     // position in the tile
    float sl2e = P.sl2e;
    f2 scale2 = pack2(sl2e, sl2e);
    uint32_t turned = 0;  // parts of this tile so far (e4m3)
    const uint32_t tO = tbase + C::TO + t * D + lane_off;
    constexpr int O0 = D / HALVES;
    bool ok = true;
    uint32_t cnt = 0;  // blocks of this tile so far
    // The second product of the latest block.  The barrier's phase before it
    // is known to be over: its S (one S buffer: S of the latest block) was
    // issued after that product.
    auto wait_product = [&]() {
      const uint32_t at = cnt - 1;
      if (ok) ok = spin_wait(&o_done[NSB == 2 ? (at & 1) : (uint32_t)t], (NSB == 2 ? at >> 1 : at) & 1, P.err);
      ok = __all_sync(0xffffffffu, ok);
    };
    // The two halves of a row trade a value; slots alternate, so that one
    // barrier a trade is enough.
    uint32_t trades = 0;
    auto trade = [&](float x) {
      float *at = xchg + (trades & 1) * 2 * ROWS;
      ++trades;
      at[hf * ROWS + r] = x;
      named_barrier(2 + (warp & 3), 64);
      return at[(hf ^ 1) * ROWS + r];
    };
    Item it{};
    if (parts > 0) it = item_at<NT>(P, pre, id_of(0));
    for (int k = 0; k < parts; ++k) {
      const Part part = part_of(k, it);
      const bool work = part.j1 > part.j0;
      if (t > 0 && it.rows <= P.PT) {  // nothing for this tile
        if (k + 1 < parts) it = item_at<NT>(P, pre, id_of(k + 1));
        continue;
      }
      const bool mine = ir < P.PT && t * P.PT + ir < it.rows;  // a row of the prompt
      const int pt = it.p0 + t * P.PT, p = pt + ir;            // position of the tile's first row, of this one
      const int plast = it.p0 + imin(it.rows, (t + 1) * P.PT) - 1;
      float m = -INFINITY, l = 0.f;
      if constexpr (F8) {
        if (work) {
          // This row of the queries (this thread's columns of it), scaled by a power of two: largest element
          // in [2^7, 2^8).  32 elements at a time, in place: their first e4m3 parts, then what those leave.
          if (ok) ok = spin_wait(&q_full[t], turned++ & 1, P.err);
          ok = __all_sync(0xffffffffu, ok);
          constexpr int PC = D / HALVES / 8;
          uint8_t *row = qs + t * C::QBYTES + r * 128;
          auto place = [&](int x) {
            x += hf * PC;
            return reinterpret_cast<uint4 *>(row + (x >> 3) * ROWS * 128 + (((x & 7) ^ (r & 7)) << 4));
          };
          uint32_t mx = 0;  // (of finite values the larger has the larger bits)
#pragma unroll 8
          for (int x = 0; x < PC; ++x) {
            const uint4 w = *place(x);
            mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
          }
          mx = max(mx & 0xffffu, mx >> 16);
          if (HALVES == 2) mx = max(mx, __float_as_uint(trade(__uint_as_float(mx))));
          const int e = (int)(mx >> 7), E = imin(imax(e, 16), 254);
          // (never 0, which would make a masked score's -inf NaN: scores this small are all 0 to their exponential)
          sl2e = fmaxf(P.sl2e * (P.ks ? P.ks[it.h] : 1.f) * __int_as_float((E - 7) << 23), 0x1p-126f);
          scale2 = pack2(sl2e, sl2e);
          float up = __int_as_float((261 - E) << 23);  // 2^(7 - (E - 127))
          if (e == 255) up = __int_as_float(0x7fffffff);  // e4m3 has no infinity: the row's scores are NaN
          const f2 up2 = pack2(up, up);
          auto two = [&](uint32_t y, uint32_t &l) {  // two elements; what the first part leaves is exact in fp16
            const float2 z = unpack2(mul2(pack2(bf16lo(y), bf16hi(y)), up2));
            const uint32_t v = pack_f16x2(z.x, z.y), h = f16x2_to_e4m3x2(v), b = e4m3x2_to_f16x2(h);
            const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&v), *reinterpret_cast<const __half2 *>(&b));
            l = f16x2_to_e4m3x2(*reinterpret_cast<const uint32_t *>(&d));
            return h;
          };
          auto four = [&](uint32_t y, uint32_t z, uint32_t &h, uint32_t &l) {
            uint32_t l0, l1;
            const uint32_t h0 = two(y, l0), h1 = two(z, l1);
            h = h0 | h1 << 16, l = l0 | l1 << 16;
          };
          // (a loop: all of it unrolled, it waits for its instructions)
#pragma unroll 1
          for (int x = 0; x < PC; x += 4) {
            uint4 w[4], hi[2], lo[2];
#pragma unroll
            for (int y = 0; y < 4; ++y) w[y] = *place(x + y);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              four(w[2 * y].x, w[2 * y].y, hi[y].x, lo[y].x);
              four(w[2 * y].z, w[2 * y].w, hi[y].y, lo[y].y);
              four(w[2 * y + 1].x, w[2 * y + 1].y, hi[y].z, lo[y].z);
              four(w[2 * y + 1].z, w[2 * y + 1].w, hi[y].w, lo[y].w);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) *place(x + y) = hi[y], *place(x + 2 + y) = lo[y];
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_ready[t]);
        }
      }
      // Both halves of a row take part in every trade whatever `ok` says (the
      // barriers have no time limit); after a wait that ran out only the work
      // is skipped.
      for (int j = part.j0; j < part.j1; ++j, ++cnt) {
        const uint32_t sb = NSB == 2 ? (cnt & 1) : (uint32_t)t;
        const uint32_t tS = tbase + C::TS + sb * BN + hf * COLS + lane_off;
        if (ok) ok = spin_wait(&s_full[sb], (NSB == 2 ? cnt >> 1 : cnt) & 1, P.err);
        ok = __all_sync(0xffffffffu, ok);
        tc::fence_after_sync();
        uint32_t raw[COLS / 32][32];
        // (after a wait that ran out what stands there has no meaning, and nothing is stored;
        // loads under a condition cost registers)
#pragma unroll
        for (int c = 0; c < COLS / 32; ++c) tc::ld32(tS + 32 * c, raw[c]);
        tc::wait_ld();
        const int base = it.base(j);
        if (base + BN - 1 > pt || (P.window > 0 && base <= plast - P.window && base + BN > P.sinks)) {
          // key c of the block is seen iff c <= hi and (c > lo or c < sk)
          const int at = base + hf * COLS, hi = p - at, lo = P.window > 0 ? hi - P.window : -1;
          const int sk = P.sinks - (j == 0 && it.ns == 0 ? hf * COLS : at);
#pragma unroll
          for (int c = 0; c < COLS / 32; ++c) {
            auto below = [&](int n) {  // bits 0..n-1 of this group of 32
              const int b = n - 32 * c;
              return b <= 0 ? 0u : b >= 32 ? 0xFFFFFFFFu : (1u << b) - 1u;
            };
            const uint32_t seen = below(hi + 1) & (~below(lo + 1) | below(sk));
#pragma unroll
            for (int e = 0; e < 32; ++e) raw[c][e] = (seen >> e & 1u) ? raw[c][e] : 0xFF800000u;  // -inf
          }
        }
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < COLS / 32; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mx4[i] = max3(mx4[i], __uint_as_float(raw[c][e + i]), __uint_as_float(raw[c][e + 4 + i]));
        float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        if (HALVES == 2) mx = fmaxf(mx, trade(mx));
        mx *= sl2e;
        float alpha = 1.f;
        if (mx > m + C::RESCALE) {
          alpha = m == -INFINITY ? 0.f : ex2_approx(m - mx);
          m = mx;
        }
        if (j > part.j0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          // the previous block's product is in O before it is rescaled
          wait_product();
          tc::fence_after_sync();
          if (ok) {
#pragma unroll 1
            for (int c0 = hf * O0; c0 < (hf + 1) * O0; c0 += 32) {
              uint32_t o[32];
              tc::ld32(tO + c0, o);
              tc::wait_ld();
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
              tc::st32(tO + c0, o);
            }
            tc::wait_st();
          }
          l *= alpha;
        }
        const float nb = m == -INFINITY ? 0.f : C::LIFT - m;
        const f2 nbase = pack2(nb, nb);
        f2 sum0 = 0, sum1 = 0;
#pragma unroll
        for (int c = 0; c < COLS / 32; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x = unpack2(fma2(pack2(__uint_as_float(raw[c][2 * e]), __uint_as_float(raw[c][2 * e + 1])),
                                          scale2, nbase));
            const float y0 = ex2_approx(x.x), y1 = ex2_approx(x.y);
            if (e & 1)
              sum1 = add2(sum1, pack2(y0, y1));
            else
              sum0 = add2(sum0, pack2(y0, y1));
            pk[e] = F8 ? pack_f16x2(y0, y1) : pack_bf16x2(y0, y1);
          }
          // over S columns that both halves have read: this half's P follows the other's
          tc::st16(tbase + C::TS + sb * BN + (hf * COLS) / 2 + 16 * c + lane_off, pk);
          if (NSB == 1 && c == COLS / 64 - 1) {
            tc::wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_half[sb]);
          }
        }
        const float2 s2 = unpack2(add2(sum0, sum1));
        l += s2.x + s2.y;
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[sb]);
      }
      const Item now = it;
      // the next item is looked up while the last product runs
      if (k + 1 < parts) it = item_at<NT>(P, pre, id_of(k + 1));
      if (work) {
        wait_product();
        tc::fence_after_sync();
      }
      if (HALVES == 2) l += trade(l);
      // O / l to bf16.  Read so that the lanes of a quad hold neighbouring
      // columns of a row; four quad lanes then trade 4-byte pieces for 16
      // consecutive bytes each, and a store covers eight rows' 64 bytes (one
      // row a lane would take 32 sectors a store).
      constexpr int NG = O0 / 64;
      if (part.j0 > 0 || part.j1 < now.n) {  // a piece of an item: O as it is, maximum and sum
        const size_t at = ((size_t)(2 * blockIdx.x + (part.j0 > 0 ? 0 : 1)) * NT + t) * ROWS + r;
        if (hf == 0 && mine && ok) P.ml[at] = make_float2(m, l);
        // four columns of all rows side by side: a warp's store is 512 bytes in one piece
        float4 *out = reinterpret_cast<float4 *>(P.opart + (at - r) * D) + (size_t)(hf * O0 / 4) * ROWS + r;
#pragma unroll 1
        for (int c = 0; c < O0 / 32; ++c) {
          uint32_t o[32];
          tc::ld32(tO + hf * O0 + 32 * c, o);
          tc::wait_ld();
          if (c == O0 / 32 - 1) {  // O is read out
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_free[t]);
          }
          if (mine && ok) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              out[(8 * c + e) * ROWS] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
          }
        }
        continue;
      }
      const float f = l != 0.f ? (F8 && P.vs ? P.vs[now.h] : 1.f) / l : 0.f;
      const long long at = (mine && ok) ? (long long)(now.q0 + t * P.PT + ir) * P.o.token_stride +
                                              (long long)(now.h * P.G + r - ir * P.G) * P.o.head_stride + hf * O0
                                        : -1LL;
      const int tq = lane & 3;
#pragma unroll 1
      for (int x0 = 0; x0 < 2 * NG; ++x0) {  // 16 rows of 64 columns at a time
        const int lh = x0 / NG, c = x0 % NG;
        uint32_t o[32];
        if (work) {
          tc::ld_16x64(tbase + C::TO + t * D + ((uint32_t)((warp & 3) * 32 + 16 * lh) << 16) + hf * O0 + 64 * c, o);
          tc::wait_ld();
          if (x0 == 2 * NG - 1) {  // O is read out
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_free[t]);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = 16 * lh + 8 * i + (lane >> 2);
          const float fr = __shfl_sync(0xffffffffu, f, row);
          const long long to = __shfl_sync(0xffffffffu, at, row);
          __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(P.o.ptr) + to + 64 * c + 8 * tq;
          const f2 fr2 = pack2(fr, fr);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int y = 16 * g + 4 * e + 2 * i;
              const float2 z = unpack2(mul2(pack2(__uint_as_float(o[y]), __uint_as_float(o[y + 1])), fr2));
              x[e] = pack_bf16x2(z.x, z.y);
            }
            auto trade4 = [&](uint32_t &lo, uint32_t &hi, int bit) {
              const bool up = tq & bit;
              const uint32_t y = __shfl_xor_sync(0xffffffffu, up ? lo : hi, bit);
              if (up) lo = y; else hi = y;
            };
            trade4(x[0], x[1], 1);
            trade4(x[2], x[3], 1);
            trade4(x[0], x[2], 2);
            trade4(x[1], x[3], 2);
            // no key seen: zeros, whatever O holds
            const uint4 v = fr != 0.f ? make_uint4(x[0], x[1], x[2], x[3]) : make_uint4(0u, 0u, 0u, 0u);
            if (to >= 0) *reinterpret_cast<uint4 *>(out + 32 * g) = v;
          }
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == C::SOFT) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tbase, 512u);
  }
}

// Joins the pieces of the item that CTA blockIdx.x begins and does not end: a warp takes 8 rows of
// 64 columns, a lane 16 columns of a row.
constexpr int JOIN_BLOCKS = 8;
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Params P, int rows) {
  pdl_wait();
  const Cut c = P.cuts[blockIdx.x];
  if (!c.pieces) return;
  const int lane = threadIdx.x & 31, n = c.pieces;
  const float vs = P.vs ? P.vs[c.h] : 1.f;
  // rows before a piece; this CTA's second, then the others' first
  auto piece = [&](int x) { return (size_t)(2 * (blockIdx.x + x) + (x == 0 ? 1 : 0)) * rows; };
#pragma unroll 1
  for (int x8 = blockIdx.y * 8 + (threadIdx.x >> 5); x8 < rows / 8 * (D / 64); x8 += JOIN_BLOCKS * 8) {
    const int row = x8 / (D / 64) * 8 + (lane & 7), c16 = x8 % (D / 64) * 16 + (lane >> 3) * 4;  // first four columns' place
    const int t = row / ROWS, r = row - t * ROWS, ir = r / P.G;
    if (ir >= P.PT || t * P.PT + ir >= c.rows) continue;
    const float4 *src = reinterpret_cast<const float4 *>(P.opart) + (size_t)t * ROWS * (D / 4) + c16 * ROWS + r;
    float m = -INFINITY, l = 0.f;
#pragma unroll 8
    for (int x = 0; x < n; ++x) m = fmaxf(m, P.ml[piece(x) + row].x);
    float4 o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int x = 0; x < n; x += 4) {
      float2 s[4];
      float4 v[4][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const size_t at = piece(imin(x + u, n - 1));
        s[u] = x + u < n ? P.ml[at + row] : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[u][e] = src[at * (D / 4) + e * ROWS];
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float w = s[u].x == -INFINITY ? 0.f : ex2_approx(s[u].x - m);
        l = fmaf(s[u].y, w, l);
        if (w == 0.f) continue;  // (a piece that the row sees nothing of holds anything)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = make_float4(fmaf(v[u][e].x, w, o[e].x), fmaf(v[u][e].y, w, o[e].y), fmaf(v[u][e].z, w, o[e].z), fmaf(v[u][e].w, w, o[e].w));
      }
    }
    const float f = l != 0.f ? vs / l : 0.f;
    uint32_t y[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y[2 * e] = f != 0.f ? pack_bf16x2(o[e].x * f, o[e].y * f) : 0u;
      y[2 * e + 1] = f != 0.f ? pack_bf16x2(o[e].z * f, o[e].w * f) : 0u;
    }
    uint4 *out = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(P.o.ptr) + (long long)(c.q0 + t * P.PT + ir) * P.o.token_stride +
                                           (long long)(c.h * P.G + r - ir * P.G) * P.o.head_stride + c16 * 4);
    out[0] = make_uint4(y[0], y[1], y[2], y[3]);
    out[1] = make_uint4(y[4], y[5], y[6], y[7]);
  }
}

// 4-D map of query rows [T][H][D] (column, head, token, 64-column group), 128-byte
// swizzle, zeros past the last token.
static bool query_map(CUtensorMap *map, const sv_rows *r, int T, int H, int D, int b1, int b2) {
  auto fn = attn::encode_fn();
  if (!fn) return false;
  // the stride of a dimension of one is never used, but has to be a valid one
  const cuuint64_t ts = T > 1 ? (cuuint64_t)r->token_stride * 2 : 128, hs = H > 1 ? (cuuint64_t)r->head_stride * 2 : 128;
  cuuint64_t dims[4] = {64, (cuuint64_t)H, (cuuint64_t)T, (cuuint64_t)(D / 64)}, strides[3] = {hs, ts, 128};
  cuuint32_t box[4] = {64, (cuuint32_t)b1, (cuuint32_t)b2, 1}, estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, r->ptr, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 5-D map of a cache (128 bytes of columns, slot, column group, head, page) in boxes of R
// slots and `groups` groups; zeros past the last page.
static bool page_map(CUtensorMap *map, void *base, const sv_paged_kv *c, int D, int Hkv, int R, int groups, bool swizzle) {
  auto fn = attn::encode_fn();
  if (!fn) return false;
  const int es = c->dtype == SV_E4M3 ? 1 : 2;
  const cuuint32_t cols = 128 / es;
  cuuint64_t dims[5] = {cols, (cuuint64_t)c->page_size, (cuuint64_t)(D * es / 128), (cuuint64_t)Hkv, (cuuint64_t)c->num_pages};
  cuuint64_t strides[4] = {(cuuint64_t)c->slot_stride * es, 128, (cuuint64_t)c->head_stride * es, (cuuint64_t)c->page_stride * es};
  cuuint32_t box[5] = {cols, (cuuint32_t)R, (cuuint32_t)groups, 1, 1}, estr[5] = {1, 1, 1, 1, 1};
  return fn(map, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, base, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int TILES, bool F8>
static sv_status run(const sv_rows *q, const sv_paged_kv *cache, Params &P, int sms, cudaStream_t s) {
  using C = Cfg<D, TILES, F8>;
  CUtensorMap mq, mk, mv;
  P.R = P.page_size % 64 == 0 ? 64 : P.page_size % 32 == 0 ? 32 : 16;
  P.piece = imax(P.R, 32);
  if (!query_map(&mq, q, P.Tq, P.Hkv * P.G, D, P.G, P.PT) || !page_map(&mk, cache->k, cache, D, P.Hkv, P.R, 1, true) ||
      !page_map(&mv, cache->v, cache, D, P.Hkv, P.R, F8 ? 1 : D / 64, !F8))
    return SV_ERR_CUDA;
  const size_t prefix = ((size_t)P.B + 1) * 4;
  P.few_slots = !F8 && prefix <= HEADER - PREFIX ? 0 : 1;
  const size_t smem = P.few_slots ? C::BEHIND + imax((int)prefix, HEADER - PREFIX) : C::RING + 160 * 1024;
  static_assert((MAX_KEPT + 1) * 16 <= HEADER - PREFIX, "sequences kept");
  static_assert(C::RING + 160 * 1024 <= 227 * 1024 && C::BEHIND + (MAX_B + 1) * 4 <= 227 * 1024, "shared memory");
  // at most one tile more per sequence than the rows fill, and no more CTAs than blocks
  P.most = P.Tq / (P.PT * C::NT) + P.B;
  const long long blocks = ((long long)P.width * P.page_size + BN - 1) / BN + 1;
  if ((long long)P.most * (blocks + HEAD_COST) > 0x7fffffffLL / P.Hkv) return SV_ERR_UNSUPPORTED;
  const int ctas = (int)lmin((long long)P.most * P.Hkv * blocks, sms);
  cudaError_t e = launch_early(chunk_attn_kernel<D, TILES, F8>, dim3(ctas), dim3(C::THREADS), smem, s, mq, mk, mv, P);
  if (e != cudaSuccess) return SV_ERR_CUDA;
  if (ctas == 1) return SV_OK;
  return from_cuda(launch_early(join_kernel<D>, dim3(ctas - 1, JOIN_BLOCKS), dim3(256), 0, s, P, C::NT * ROWS));
}

template <bool F8>
static sv_status run_any(const sv_rows *q, const sv_paged_kv *cache, Params &P, int D, int sms, cudaStream_t s) {
  if (D == 256) return run<256, 1, F8>(q, cache, P, sms, s);
  // Two tiles a CTA share each block of keys; they pay where most sequences fill more than
  // one.
  return P.Tq > (long long)P.B * P.PT ? run<128, 2, F8>(q, cache, P, sms, s) : run<128, 1, F8>(q, cache, P, sms, s);
}

// Pieces of cut items: two a CTA.
static size_t part_rows(int D) { return (size_t)(D == 128 ? 2 : 1) * ROWS; }
static size_t pieces_bytes(int sms, int D) { return 2 * (size_t)sms * part_rows(D) * ((size_t)D * 4 + 8); }

}  // namespace chunk
}  // namespace sv

using namespace sv;

extern "C" {

size_t paged_chunk_attn_workspace_bytes(int B, int Tq, int Hq, int Hkv, int D) {
  (void)Hq, (void)Hkv;
  const int sms = device_sm_count();
  if (B < 1 || Tq < 1 || (D != 128 && D != 256) || sms <= 0) return 0;
  return chunk::pieces_bytes(sms, D) + (size_t)sms * sizeof(chunk::Cut);
}

sv_status paged_chunk_attn(const sv_rows *q, const sv_paged_kv *cache, const int32_t *block_table, int64_t table_stride,
                           int table_width, const int32_t *kv_lens, const sv_rows *o, const int32_t *cu_q, int B, int Tq,
                           int Hq, int Hkv, int D, float scale, int window, int sinks, void *workspace, size_t ws_bytes,
                           sv_stream_t stream) {
  if (B < 0 || Tq < 0 || Hq < 1 || Hkv < 1 || D < 1 || Hq % Hkv != 0) return SV_ERR_INVALID_ARG;
  if (window < 0 || sinks < 0 || table_width < (B > 0 ? 1 : 0) || table_stride < 0) return SV_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !(scale < INFINITY)) return SV_ERR_INVALID_ARG;
  if (D != 128 && D != 256) return SV_ERR_UNSUPPORTED;
  const int G = Hq / Hkv;
  if (G > chunk::ROWS || B > chunk::MAX_B || Tq > 0x40000000 || window > 0x40000000) return SV_ERR_UNSUPPORTED;
  if (!paged::good_rows(q, Tq) || !paged::good_rows(o, Tq)) return SV_ERR_INVALID_ARG;
  const sv_status cs = paged::check_cache(cache, D);
  if (cs != SV_OK) return cs;
  if (B > 0 && (!block_table || !kv_lens || !cu_q)) return SV_ERR_INVALID_ARG;
  if (!paged::aligned(block_table, 4) || !paged::aligned(kv_lens, 4) || !paged::aligned(cu_q, 4)) return SV_ERR_INVALID_ARG;
  if ((long long)table_width * cache->page_size > 0x40000000LL) return SV_ERR_UNSUPPORTED;
  if (B == 0 || Tq == 0) return SV_OK;
  // a tensor map steps by every stride: rows that repeat (stride 0) have none
  if ((Tq > 1 && !q->token_stride) || (Hq > 1 && !q->head_stride)) return SV_ERR_UNSUPPORTED;
  const int sms = device_sm_count();
  if (sms <= 0) return SV_ERR_CUDA;
  if (!workspace || ws_bytes < paged_chunk_attn_workspace_bytes(B, Tq, Hq, Hkv, D)) return SV_ERR_WORKSPACE;
  if (!paged::aligned(workspace, 16)) return SV_ERR_INVALID_ARG;
  chunk::Params P{};
  P.o = *o;
  P.cu_q = cu_q, P.lens = kv_lens, P.table = block_table, P.table_stride = table_stride;
  P.width = table_width, P.page_size = cache->page_size, P.num_pages = (int)cache->num_pages;
  P.ks = cache->k_scale, P.vs = cache->v_scale;
  P.opart = static_cast<float *>(workspace);
  P.ml = reinterpret_cast<float2 *>(P.opart + 2 * (size_t)sms * chunk::part_rows(D) * D);
  P.cuts = reinterpret_cast<chunk::Cut *>(static_cast<uint8_t *>(workspace) + chunk::pieces_bytes(sms, D));
  P.err = device_error_word();
  if (!P.err) return SV_ERR_CUDA;
  P.B = B, P.Tq = Tq, P.Hkv = Hkv, P.G = G, P.PT = chunk::ROWS / G;
  P.sl2e = scale * 1.4426950408889634f;
  P.window = window, P.sinks = sinks;
  P.stall = launch_flags() & SV_LAUNCH_TEST_STALL_COPY ? 1 : 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return cache->dtype == SV_E4M3 ? chunk::run_any<true>(q, cache, P, D, sms, s) : chunk::run_any<false>(q, cache, P, D, sms, s);
}

}  // extern "C"
