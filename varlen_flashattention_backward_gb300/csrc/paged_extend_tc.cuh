// fa_paged_extend for 16-bit types on the sm_103a tensor cores (tcgen05 with
// accumulators in TMEM, TMA loads).  Included by one translation unit per type.
//
// A block is 256 packed query rows, two halves of 128, one for each of two softmax
// warpgroups; a tile is BN = 128 keys (64 at head dim 192, whose accumulators fill
// TMEM).  Per tile and half:
//
//   S  = Q K^T    M = 128 rows, N = BN keys, K = D   (Q, K in shared memory, K-major)
//   O += P V      M = 128 rows, N = D, K = BN keys   (P in TMEM over S, V MN-major)
//
// The halves take turns on the tensor core, so that one half's products run during the
// other's softmax.  Where a block has 128 rows or fewer (single tokens, drafts, the end
// of a chunk), both warpgroups take the same rows and every other tile each, and their
// results are added in the end: the same pipeline, with twice the keys on the way.
//
// Warps: 0-3 and 4-7 softmax (a thread is a row), 8 loads K, walks the CTA's span and
// tells the others what comes next, 9 issues the MMAs, 10 loads V, 11 Q.
//
// The running maximum is replaced only where it has grown by more than 2^8: weights
// then pass 1, by that much at most, and the accumulators are seldom read back.  Weights
// are rounded to the type for the second product: half a step of the type relative
// to each weight, of the size of y's own rounding; their sum is taken before.  fp16
// weights carry 2^7, so that 2^8 of them still fits and 2^-31 of a row's largest
// is still held.  bf16 weights carry 2^-8 and so never pass 1: sums of products leave
// fp32's range only where those of exp(S - max) would.
//
// Every wait is bounded; one that gives up sets FA_PAGED_TIMEOUT, and the CTA winds down
// without waits but for its own copies and MMAs in flight.
//
// 2048 tokens behind 30000, 32 heads on 8, D 128, bf16: 635 us, 1640 TFLOP/s, for the first
// 60 ms at full clocks (87% of the measured burst peak), and 702 us, 1480 TFLOP/s, from
// then on, under the power cap (87% of the sustained one).  A turn of both halves takes 2900 cycles, their products 2048; what is
// left is the way of a half from scores over softmax and products to its next scores,
// which two halves cannot hide altogether.  Instruction fetches were the largest stall
// of all: with the two halves of a tile unrolled the loop took 710 us, hence one copy of
// the code per purpose, and rare paths out of line.  64 drafts of 5 tokens over 1024 to
// 8192 keys: 218 us, 6.0 TB/s, 88% of the copy bandwidth.  At D 64 and 32 the softmax
// bounds it (the first case 527 us at D 64, 2600 cycles a turn, 1024 of them
// exponentials).

#include <cuda.h>

#include <type_traits>

#include "paged_extend.cuh"

namespace fav {
namespace {

using namespace sm103;

constexpr int kBR = 256;
constexpr int kThreads = 384;
constexpr int kControl = 3 << 10;      // bytes for the control block
constexpr float kLazy = 8.f;      // log2 of how far the maximum may grow past the one in use

struct ExtendMaps {
  CUtensorMap k, v, q;
  int box;            // keys of a copy; 0: pages that TMA cannot take
  int token_first;    // axes 1 and 2 are tokens and heads, not heads and tokens
  int by_tma;         // so are the query rows
};

template <int D_>
struct Dim {
  static constexpr int D = D_;
  static constexpr int BN = D > 128 ? 64 : 128;
  static constexpr int kPanels = (D + 63) / 64;           // of 64 columns, 128-byte rows
  static constexpr int kPanel = BN * 128;                 // of K or V
  static constexpr int kStage = kPanels * kPanel;
  static constexpr int kQPanel = 128 * 128;
  static constexpr int kQ = kPanels * kQPanel;            // of one half
  static constexpr int fit() {
    const int s = (232448 - kControl - 2 * kQ) / kStage;
    return s < 8 ? s : 8;
  }
  static constexpr int kStages = fit();
  // Of K, which a product frees at once, and of V, which waits for the softmax.
  static constexpr int kStagesK = kStages / 2, kStagesV = kStages - kStagesK;
  static constexpr int kSmem = 2 * kQ + kStages * kStage + kControl;
  static_assert(kStages >= 4 && kStages * kStage >= int(sizeof(Measure)), "shared memory");
  // TMEM columns.  Where there is room the weights have columns of their own, so that
  // the next scores can be computed as soon as a tile's have been read; else they take
  // the scores' place.
  static constexpr bool kAhead = D <= 64;
  __host__ __device__ static constexpr uint32_t s_col(int w) { return uint32_t(w * BN); }
  __host__ __device__ static constexpr uint32_t o_col(int w) {
    return uint32_t(2 * BN + w * (D > 128 ? D : D > 64 ? 128 : 64));
  }
  __host__ __device__ static constexpr uint32_t p_col(int w) { return kAhead ? uint32_t(384 + w * 64) : s_col(w); }
  static_assert(2 * BN + 2 * (D > 128 ? D : 128) <= 512, "TMEM");
};

// Where a tile of the CTA's is: its stage, and how often that was used before.
struct Stage {
  int stage, turn;
};
template <int D>
__device__ __forceinline__ Stage place_of(int kv, int tile) {
  using M = Dim<D>;
  if (kv) return {M::kStagesK + tile % M::kStagesV, tile / M::kStagesV};
  return {tile % M::kStagesK, tile / M::kStagesK};
}

// What the walking warp tells the others of a segment.
struct Item {
  Request r;
  int row0, rows;      // packed rows
  int b, h, key0, steps;  // first key of its first tile; turns of a softmax warpgroup, both together
  int both;            // the halves have rows of their own
  int tile;            // number of its first tile in the CTA
  int slot, item, first, end;
};

constexpr int kMasks = 16;    // tiles whose key masks are held
constexpr int kItems = 4;     // segments handed out at a time

struct Control {
  uint64_t full[8], empty[8], ready[2], taken[2], weights[2][2], half[2], spent[2], query[2], query_free[2], item_full[kItems], item_empty[kItems], done, read, last;
  // ready: scores; taken: they have been read; weights: of a half of the keys; half, spent:
  // the products of those halves with the values are done.
  uint32_t tmem;
  int abort, flagged, odd;
  Item item[kItems];
  alignas(16) uint32_t mask[kMasks][4];   // which keys' pages are the cache's
  float part[3][128];                     // the second half's sums of a shared block
  Record record;
};
static_assert(sizeof(Control) <= kControl, "control block");

struct Ctl {
  int *abort;
  int32_t *error;
  long long timeout;
};

// Keeps code that seldom runs out of the loops' way: what the instruction caches hold is
// little more than those.
__device__ __forceinline__ bool unlikely(bool x) { return __builtin_expect(x, false); }

// By a whole warp; the same for all of it.
__device__ __forceinline__ bool wait_on(const Ctl &c, uint32_t bar, uint32_t parity) {
  if (__all_sync(kFull, mbar_wait(bar, parity, c.timeout, c.abort))) return true;
  if (!*reinterpret_cast<volatile int *>(c.abort)) {
    *reinterpret_cast<volatile int *>(c.abort) = 1;
    if (c.error) atomicOr(c.error, FA_PAGED_TIMEOUT);
  }
  return false;
}
__device__ __forceinline__ bool wait(const Ctl &c, uint32_t bar, uint32_t parity) {
  return unlikely(!__all_sync(kFull, mbar_try_wait(bar, parity))) ? wait_on(c, bar, parity) : true;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// `bar` waits for this thread's copies so far: its count goes up by one now and down by
// one when they are there.  Ahead of the arrival that would complete the phase.
__device__ __forceinline__ void cp_async_count_in(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y,
                                            int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y,
                                            int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t ta, const uint32_t (&r)[32]) {
  uint32_t a[16], b[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    a[i] = r[i];
    b[i] = r[16 + i];
  }
  tmem_st16(ta, a);
  tmem_st16(ta + 16, b);
}

// A load of 32 columns in two steps: between them the registers hold nothing.
__device__ __forceinline__ void tmem_ld32_start(uint32_t ta, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(ta)
      : "memory");
}
// (The registers pass through it, so that no use of them moves ahead of the wait.)
__device__ __forceinline__ void tmem_ld32_end(uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
        "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
        "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),
        "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
        "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]),
        "+r"(r[31])
      :
      : "memory");
}

__device__ __forceinline__ void add2(float &x, float &y, float a, float b) {
  asm("{\n\t.reg .b64 s, t;\n\tmov.b64 s, {%0, %1};\n\tmov.b64 t, {%2, %3};\n\t"
      "add.rn.f32x2 s, s, t;\n\tmov.b64 {%0, %1}, s;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return std::is_same<T, __nv_bfloat16>::value ? pack_bf16(lo, hi) : pack_f16(lo, hi);
}

// Trades 16 bytes with the lane beside.
__device__ __forceinline__ uint4 trade(uint4 v) {
  return make_uint4(__shfl_xor_sync(kFull, v.x, 1), __shfl_xor_sync(kFull, v.y, 1), __shfl_xor_sync(kFull, v.z, 1),
                    __shfl_xor_sync(kFull, v.w, 1));
}

// ---------------------------------------------------------------------------
// Loaders, one warp for K and one for V
// ---------------------------------------------------------------------------
// Each has a ring of its own: tile i of the CTA's is in its place i.  A tile whose pages
// are all good and whole comes by TMA, in boxes of as many keys as divide page and
// tile; the last one of a request, one with a bad page, and pages of other sizes come
// in 16-byte pieces, zeros for what is not there.  Nothing here waits for a copy: the
// stage's barrier counts the pieces in, and their reader, the MMA warp, makes the proxy
// fence that they need.
template <typename T, int D>
struct Loader {
  using M = Dim<D>;
  static constexpr int kRows = M::BN / 32;   // keys per lane
  const ExtendParams &p;
  const ExtendMaps &maps;
  Control *c;
  uint32_t ring;
  Ctl ctl;
  int lane, kv;                        // kv: 0 for K, 1 for V
  bool odd = false;                    // some key has a bad page
  int tiles = 0;                       // so far

  __device__ __forceinline__ uint32_t bar(uint64_t &b) const { return smem_u32(&b); }

  // The page of key `key` of request b, or -1.
  __device__ __forceinline__ int page_of(int b, int key, int len) const {
    if (key >= len) return -1;
    return p.table[b * p.table_stride + (p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size)];
  }
  __device__ __forceinline__ int token_of(int key) const {
    return p.page_shift >= 0 ? key & (p.page_size - 1) : key % p.page_size;
  }

  // What a tile's loads need of the table, looked up one tile ahead: the page of this
  // lane's box, or those of the keys lane, lane + 32, ...
  struct Pages {
    int of[kRows];
  };
  __device__ __forceinline__ bool boxed(int len, int key0) const {
    return maps.box != 0 && key0 + M::BN <= len;
  }
  __device__ __forceinline__ Pages look_up(int len, int b, int key0) const {
    Pages pages;
    if (boxed(len, key0)) {
      pages.of[0] = page_of(b, key0 + (lane & (M::BN / maps.box - 1)) * maps.box, len);
    } else {
#pragma unroll
      for (int k = 0; k < kRows; ++k) pages.of[k] = page_of(b, key0 + k * 32 + lane, len);
    }
    return pages;
  }

  __device__ __forceinline__ bool tile(int len, int b, int h, int key0, const Pages &pages) {
    const int which = tiles & (kMasks - 1);
    const Stage place = place_of<D>(kv, tiles);
    if (place.turn > 0 && !wait(ctl, bar(c->empty[place.stage]), uint32_t(place.turn - 1) & 1)) return false;
    ++tiles;
    const uint32_t full = bar(c->full[place.stage]);
    const bool box = boxed(len, key0);
    if (box && __all_sync(kFull, pages.of[0] >= 0 && pages.of[0] < p.num_pages)) {
      const int boxes = M::BN / maps.box, mine = lane & (boxes - 1);
      const int token = token_of(key0 + mine * maps.box);
      if (kv == 0 && lane < 4) c->mask[which][lane] = ~0u;
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(full, M::kStage);
      __syncwarp();
      const uint32_t dst = ring + place.stage * M::kStage + mine * maps.box * 128;
      const CUtensorMap *map = kv ? &maps.v : &maps.k;
      for (int pl = lane / boxes; pl < M::kPanels; pl += 32 / boxes)
        tma_load_4d(dst + pl * M::kPanel, map, full, pl * 64, maps.token_first ? token : h,
                    maps.token_first ? h : token, pages.of[0]);
      __syncwarp();
      return true;
    }
    // A row's 16-byte pieces go to kAcross neighbouring lanes, the rows of 32 keys one
    // after the other.
    constexpr int kChunks = D / 8;
    constexpr int kAcross = kChunks <= 4 ? 4 : kChunks <= 8 ? 8 : kChunks <= 16 ? 16 : 32;
    const T *cache = static_cast<const T *>(kv ? p.vc : p.kc);
    const int ch = lane & (kAcross - 1), sub = lane / kAcross;
    const uint32_t dst = ring + place.stage * M::kStage + (ch >> 3) * M::kPanel;
    int good = 0;
#pragma unroll 1
    for (int k = 0; k < kRows; ++k) {
      const int key = key0 + k * 32 + lane;
      // (A tile that boxes would have taken but for a bad page looks its keys up here.)
      const int page = box ? page_of(b, key, len)
                           : kRows == 2 ? (k == 0 ? pages.of[0] : pages.of[1])
                                        : k == 0   ? pages.of[0]
                                          : k == 1 ? pages.of[1]
                                          : k == 2 ? pages.of[kRows - 2]
                                                   : pages.of[kRows - 1];
      int64_t at = -1;     // of the key's row in the cache (keys behind the request's have page -1)
      if (page >= 0 && page < p.num_pages)
        at = page * p.page_stride + token_of(key) * p.token_stride + h * p.head_stride;
      const uint32_t word = __ballot_sync(kFull, at >= 0);
      good += __popc(word);
      if (kv == 0 && lane == 0) c->mask[which][k] = word;
#pragma unroll 4
      for (int r0 = 0; r0 < 32; r0 += 32 / kAcross) {
        const int r = r0 + sub;
        const int64_t from = __shfl_sync(kFull, at, r);
        if (ch < kChunks)
          cp_async16(dst + (k * 32 + r) * 128 + (((ch & 7) ^ (r & 7)) << 4),
                     cache + (from >= 0 ? from + ch * 8 : 0), from >= 0);
      }
    }
    odd |= good < min(len - key0, M::BN);
    if (box) {      // the MMA warp does not expect pieces here
      cp_async_wait_all();
      fence_proxy_async_smem();
    } else {
      cp_async_count_in(full);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(full);
    return true;
  }

  // All tiles of a segment.
  __device__ __forceinline__ bool all(int len, int b, int h, int key0, int count) {
    Pages pages = look_up(len, b, key0);
    for (int t = 0; t < count; ++t) {
      Pages next = pages;
      if (t + 1 < count) next = look_up(len, b, key0 + (t + 1) * M::BN);
      if (!tile(len, b, h, key0 + t * M::BN, pages)) return false;
      pages = next;
    }
    return true;
  }

  // No copy may still be writing shared memory when the CTA exits, nor the arrival that
  // counts pieces in, which comes behind them.
  __device__ __forceinline__ void drain(long long ns) {
    cp_async_wait_all();
    const int never = 0, stages = kv ? M::kStagesV : M::kStagesK;
    for (int t = tiles > stages ? tiles - stages : 0; t < tiles; ++t) {
      const Stage at = place_of<D>(kv, t);
      mbar_wait(bar(c->full[at.stage]), uint32_t(at.turn) & 1, ns, &never);
    }
  }
};

// N MMAs one after the other, by the lane that is elected once for all of them.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void mma_steps(F &&f, uint32_t leader) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{}, leader);
    mma_steps<N, I + 1>(f, leader);
  }
}
template <int N, typename F>
__device__ __forceinline__ void mma_row(F &&f) {
  uint32_t leader;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(leader));
  mma_steps<N>(f, leader);
}
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t adds) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\tsetp.ne.b32 e, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(adds), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t adds) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\tsetp.ne.b32 e, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(adds), "r"(leader)
      : "memory");
}

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    extend_tc_kernel(const __grid_constant__ ExtendParams p, const __grid_constant__ ExtendMaps maps) {
  using M = Dim<D>;
  constexpr int BN = M::BN;
  constexpr bool kBF16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr float kBias = kBF16 ? kExtendBiasBf16 : kExtendBiasFp16;      // log2 of what weights carry
  static_assert(!kBF16 || kBias == -kLazy, "bf16 weights stop at 1");
  extern __shared__ __align__(1024) uint8_t sm[];     // (a swizzle atom)
  Control *c = reinterpret_cast<Control *>(sm + 2 * M::kQ + M::kStages * M::kStage);
  const uint32_t sq = smem_u32(sm), ring = sq + 2 * M::kQ;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFull, tid >> 5, 0);
  const auto bar = [](uint64_t &b) { return smem_u32(&b); };
  Ctl ctl{&c->abort, p.error, p.wait_ns};
  // Waits for this CTA's own copies and MMAs, which finish without help.
  const long long drain_ns = p.wait_ns > 1000000000LL ? p.wait_ns : 1000000000LL;

  if (tid == 0) {
    c->abort = c->flagged = c->odd = 0;
    for (int i = 0; i < M::kStages; ++i) {
      mbar_init(bar(c->full[i]), 1);
      mbar_init(bar(c->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(c->ready[i]), 1);
      mbar_init(bar(c->taken[i]), 4);
      mbar_init(bar(c->half[i]), 1);
      mbar_init(bar(c->spent[i]), 1);
      mbar_init(bar(c->weights[i][0]), 4);
      mbar_init(bar(c->weights[i][1]), 4);
      mbar_init(bar(c->query[i]), 1);
      mbar_init(bar(c->query_free[i]), 4);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(bar(c->item_full[i]), 1);
      mbar_init(bar(c->item_empty[i]), 12);
    }
    mbar_init(bar(c->done), 4);
    mbar_init(bar(c->read), 4);
    mbar_init(bar(c->last), 1);
    mbar_fence_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&c->tmem), 512);
    tmem_relinquish();
  }
  Line line;
  Place at;
  const bool any = measure<kBR, BN, kThreads>(p, *reinterpret_cast<Measure *>(sm + 2 * M::kQ), line, at);
  asm volatile("griddepcontrol.launch_dependents;");
  fence_proxy_async_smem();       // the scratch becomes the ring
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem;

  if (warp >= 8) {
    // 2 x 128 x 208 + 128 x 88 = 64512 registers, as launched (384 x 168).
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8 || warp == 10) {
      // ---------------------------------------------------------------- K and the walk, V
      Loader<T, D> load{p, maps, c, ring, ctl, lane, warp == 8 ? 0 : 1};
      Walk<kBR, BN> walk;
      walk.begin(p, line, at, any);
      for (uint32_t items = 0;; ++items) {
        const int slot = int(items % kItems);
        Item &it = c->item[slot];
        if (warp == 8) {
          Segment seg;
          const bool more = walk.next(p, seg);
          if (items >= kItems && !wait(ctl, bar(c->item_empty[slot]), (items / kItems - 1) & 1)) break;
          if (lane == 0) {
            it.end = !more;
            if (more) {
              it.r = seg.r;
              it.row0 = seg.k.row0;
              it.rows = seg.k.rows;
              it.b = seg.b;
              it.h = seg.h;
              it.key0 = (seg.k.tile0 + seg.t0) * BN;
              it.both = seg.k.rows > 128;
              it.steps = (seg.t1 - seg.t0) << it.both;
              it.tile = load.tiles;
              it.slot = seg.slot;
              it.item = seg.item;
              it.first = seg.t0 == 0;
            }
            mbar_arrive(bar(c->item_full[slot]));
          }
          __syncwarp();
        } else if (!wait(ctl, bar(c->item_full[slot]), (items / kItems) & 1)) {
          break;
        }
        const int len = it.r.len, b = it.b, h = it.h, key0 = it.key0, end = it.end, count = it.steps >> it.both;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(c->item_empty[slot]));
        if (end || !load.all(len, b, h, key0, count)) break;
      }
      if (load.odd && lane == 0) c->odd = 1;
      load.drain(drain_ns);
      if (warp == 8 && lane == 0) c->record = walk.rec;
    } else if (warp == 11) {
      // ---------------------------------------------------------------- Q
      // A warpgroup frees its rows when it has its last scores; rows that both use, when
      // both have.
      constexpr int kChunks = D / 8;
      uint32_t freed[2] = {0, 0};        // how often each warpgroup has, or will have
      uint32_t filled[2] = {0, 0};       // how often copies to each half have begun
      bool shared = false;
      for (uint32_t items = 0;; ++items) {
        const int slot = int(items % kItems);
        if (!wait(ctl, bar(c->item_full[slot]), (items / kItems) & 1)) break;
        const Item it = c->item[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(c->item_empty[slot]));
        if (it.end) break;
        if (it.steps == 0) continue;
        // They have to wait for the rows before them, but may come as far as the L2.
        if (maps.by_tma && lane < M::kPanels << it.both)
          tma_prefetch_l2_3d(&maps.q, (lane >> it.both) * 64, it.h * p.group,
                             it.r.start + (it.row0 + (lane & it.both) * 128) / p.group);
        bool ok = true;
        for (int w = 0; ok && w < (it.both ? 2 : 1); ++w) {
          if (freed[w] > 0) ok = wait(ctl, bar(c->query_free[w]), (freed[w] - 1) & 1);
          if (ok && w == 0 && shared) ok = wait(ctl, bar(c->query_free[1]), (freed[1] - 1) & 1);
          if (!ok) break;
          ++filled[w];     // now: the other half's wait may give up while these copies are on the way
          const uint32_t dst = sq + w * M::kQ;
          if (maps.by_tma) {
            // 128 / group tokens and the group's heads are 128 packed rows; what lies behind
            // the request is loaded too, and not used.
            if (lane == 0) {
              mbar_arrive_expect_tx(bar(c->query[w]), M::kQ);
              for (int pl = 0; pl < M::kPanels; ++pl)
                tma_load_3d(dst + pl * M::kQPanel, &maps.q, bar(c->query[w]), pl * 64, it.h * p.group,
                            it.r.start + (it.row0 + w * 128) / p.group);
            }
            __syncwarp();
            continue;
          }
          constexpr int kAcross = kChunks <= 4 ? 4 : kChunks <= 8 ? 8 : kChunks <= 16 ? 16 : 32;
          const int ch = lane & (kAcross - 1), sub = lane / kAcross;
#pragma unroll 1
          for (int r0 = 0; r0 < 128; r0 += 32) {
            // Neighbouring lanes take neighbouring pieces of a row; zeros behind the last.
            const int in_block = w * 128 + r0 + lane, packed = it.row0 + in_block;
            const int t = packed / p.group, n = it.h * p.group + packed - t * p.group;
            const int64_t own = in_block < it.rows ? (it.r.start + t) * p.q_stride + int64_t(n) * D : -1;
#pragma unroll 2
            for (int r1 = 0; r1 < 32; r1 += 32 / kAcross) {
              const int r = r1 + sub;
              const int64_t from = __shfl_sync(kFull, own, r);
              if (ch >= kChunks) continue;
              const uint32_t to = dst + (ch >> 3) * M::kQPanel + (r0 + r) * 128 + (((ch & 7) ^ (r & 7)) << 4);
              const uint16_t *e = static_cast<const uint16_t *>(p.q) + (from >= 0 ? from + ch * 8 : 0);
              if (p.q_chunks) {
                cp_async16(to, e, from >= 0);
              } else {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (from >= 0)
                  v = make_uint4(e[0] | uint32_t(e[1]) << 16, e[2] | uint32_t(e[3]) << 16,
                                 e[4] | uint32_t(e[5]) << 16, e[6] | uint32_t(e[7]) << 16);
                st_shared_v4(to, v);
              }
            }
          }
          if (p.sign == 1 && p.q_chunks) {
            cp_async_count_in(bar(c->query[w]));
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(c->query[w]));
            continue;
          }
          cp_async_wait_all();
          if (p.sign != 1) {       // each lane its own pieces
            const uint32_t flip = p.sign < 0 ? 0x80008000u : 0u, keep = p.sign == 0 ? 0u : ~0u;
#pragma unroll 1
            for (int r = sub; r < 128; r += 32 / kAcross) {
              if (ch >= kChunks) continue;
              uint4 *at = reinterpret_cast<uint4 *>(sm + w * M::kQ + (ch >> 3) * M::kQPanel + r * 128 +
                                                    (((ch & 7) ^ (r & 7)) << 4));
              const uint4 v = *at;
              *at = make_uint4((v.x ^ flip) & keep, (v.y ^ flip) & keep, (v.z ^ flip) & keep,
                               (v.w ^ flip) & keep);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(c->query[w]));
        }
        if (!ok) break;
        shared = !it.both && it.steps > 1;
        ++freed[0];
        if (it.steps > 1) ++freed[1];
      }
      // As Loader::drain.
      cp_async_wait_all();
      const int never = 0;
      for (int w = 0; w < 2; ++w)
        if (filled[w] > 0) mbar_wait(bar(c->query[w]), (filled[w] - 1) & 1, drain_ns, &never);
    } else if (warp == 9) {
      // ---------------------------------------------------------------- MMA issuer
      const uint32_t id_s = idesc_f16(128, BN, false, false, kBF16);
      const uint32_t id_o = idesc_f16(128, D, false, true, kBF16);
      // What the MMAs' operands are made of is the same in all lanes, and the compiler has
      // to see that: it then stays in uniform registers, and MMAs follow one another
      // without gaps (95 and more cycles an MMA otherwise, for 64).
      const uint64_t q_desc = sdesc_sw128(sq, 16, 1024);
      const uint64_t k_desc = sdesc_sw128(ring, 16, 1024), v_desc = sdesc_sw128(ring, M::kPanel, 1024);
      int k_stage = 0, v_stage = M::kStagesK;
      uint32_t k_turn = 0, v_turn = 0, weights_turn[2] = {0, 0}, query_turn[2] = {0, 0};
      uint32_t taken_turn[2] = {0, 0};
      // Where tiles come in 16-byte pieces: all, or the last one of a request.
      const bool pieces = maps.box == 0;
      bool ok = true;
      // S of the next tile for half w; `frees`: the last use of its K.
      const auto scores = [&](auto half, bool own, bool frees, bool last) {
        constexpr int w = decltype(half)::value;
        if (!wait(ctl, bar(c->full[k_stage]), k_turn)) return false;
        if (pieces || last) fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t a = q_desc + (own ? (w * M::kQ) >> 4 : 0);
        const uint64_t b = k_desc + ((k_stage * M::kStage) >> 4);
        mma_row<D / 16>([&](auto step, uint32_t leader) {
          constexpr int kk = decltype(step)::value;
          mma_ss(leader, tmem + M::s_col(w), a + (((kk >> 2) * M::kQPanel + (kk & 3) * 32) >> 4),
                 b + (((kk >> 2) * M::kPanel + (kk & 3) * 32) >> 4), id_s, kk > 0 ? 1u : 0u);
        });
        mma_commit_w(bar(c->ready[w]));
        if (frees) {
          mma_commit_w(bar(c->empty[k_stage]));
          if (++k_stage == M::kStagesK) k_stage = 0, k_turn ^= 1;
        }
        return true;
      };
      const auto values = [&](auto half, uint32_t adds, bool frees, bool last) {
        constexpr int w = decltype(half)::value;
        if (!wait(ctl, bar(c->full[v_stage]), v_turn)) return false;
        if (pieces || last) fence_proxy_async_smem();
        const uint64_t b = v_desc + ((v_stage * M::kStage) >> 4);
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          if (!wait(ctl, bar(c->weights[w][part]), weights_turn[w])) return false;
          tc_fence_after();
          mma_row<BN / 32>([&](auto step, uint32_t leader) {
            constexpr int kk = decltype(step)::value;
            const int k = part * (BN / 32) + kk;
            mma_ts(leader, tmem + M::o_col(w), tmem + M::p_col(w) + k * 8, b + ((k * 2048) >> 4), id_o,
                   kk > 0 ? 1u : adds | part);
          });
          mma_commit_w(bar(part == 0 ? c->half[w] : c->spent[w]));
        }
        weights_turn[w] ^= 1;
        if (frees) {
          mma_commit_w(bar(c->empty[v_stage]));
          if (++v_stage == M::kStages) v_stage = M::kStagesK, v_turn ^= 1;
        }
        return true;
      };
      const auto query = [&](int w) {
        const bool there = wait(ctl, bar(c->query[w]), query_turn[w]);
        query_turn[w] ^= 1;
        if (!maps.by_tma) fence_proxy_async_smem();
        return there;
      };
      constexpr std::integral_constant<int, 0> first{};
      constexpr std::integral_constant<int, 1> second{};
      for (uint32_t items = 0; ok; ++items) {
        const int slot = int(items % kItems);
        if (!wait(ctl, bar(c->item_full[slot]), (items / kItems) & 1)) break;
        const Item &it = c->item[slot];
        const int steps = __shfl_sync(kFull, it.steps, 0);
        const bool both = __shfl_sync(kFull, it.both, 0) != 0, end = __shfl_sync(kFull, it.end, 0) != 0;
        const bool tail = __shfl_sync(kFull, it.key0 + (steps >> it.both) * BN > it.r.len, 0);
        if (end) break;
        if (lane == 0) mbar_arrive(bar(c->item_empty[slot]));
        __syncwarp();
        if (steps == 0) continue;
        // One turn of a half: the products with the values of step s, and before or behind
        // them the scores of its next step.  The first turns have no values yet.
        const auto turn = [&](auto half, int s, bool frees) {
          constexpr int w = decltype(half)::value;
          if (M::kAhead && s >= 0) {
            if (!wait(ctl, bar(c->taken[w]), taken_turn[w])) return false;
            taken_turn[w] ^= 1;
          }
          const bool last = tail && s + 2 >= steps;
          if (!M::kAhead && s >= 0 && !values(half, s >= 2, frees, last)) return false;
          if (s + 2 < steps) {
            if (s < 0 && (w == 0 || both) && !query(w)) return false;
            if (!scores(half, both, frees, tail && s + 4 >= steps)) return false;
          }
          return !M::kAhead || s < 0 || values(half, s >= 2, frees, last);
        };
        for (int s = -2; ok && s < steps; s += 2) {
          ok = turn(first, s, !both);
          if (ok && s + 1 < steps) ok = turn(second, s + 1, true);
        }
      }
      // Every MMA has finished before TMEM is freed.
      mma_commit_w(bar(c->last));
      const int never = 0;
      mbar_wait(bar(c->last), 0, drain_ns, &never);
    }
  } else {
    // ------------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int w = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lanes = uint32_t(quarter * 32) << 16;
    const uint32_t t_s = tmem + lanes + M::s_col(w), t_o = tmem + lanes + M::o_col(w);
    const uint32_t t_p = tmem + lanes + M::p_col(w);
    const float scale = p.scale_log2;
    uint32_t tiles = 0, shared_at = 0;       // worked off so far
    for (uint32_t items = 0;; ++items) {
      // What is needed of the item in the end is read again then, so that the loop has
      // its registers for scores.
      const int slot = int(items % kItems);
      if (!wait(ctl, bar(c->item_full[slot]), (items / kItems) & 1)) break;
      const Item &it = c->item[slot];
      if (it.end) break;
      const auto release = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(c->item_empty[slot]));
      };
      const bool both = it.both;
      const int in_block = both ? w * 128 + row : row;
      const bool mine = in_block < it.rows;
      int lo = 0, hi = 0x7fffffff;      // rows that are not there are not masked, and not written
      if (mine) keys_of(p, it.r, (it.row0 + in_block) / p.group, lo, hi);
      const int turns = both ? it.steps / 2 : (it.steps + 1 - w) / 2;
      float m = -CUDART_INF_F, top = -CUDART_INF_F, l = 0.f;   // m: the maximum in use
      bool ok = true;
      const int stride = both ? 1 : 2;
      int k0 = it.key0 + (both ? 0 : w * BN), which = it.tile + (both ? 0 : w);
      for (int i = 0; i < turns; ++i, ++tiles, k0 += stride * BN, which += stride) {
        if (!(ok = wait(ctl, bar(c->ready[w]), tiles & 1))) break;
        tc_fence_after();
        constexpr int kHalf = BN / 64;
        uint32_t s[kHalf][32];
#pragma unroll
        for (int j = 0; j < kHalf; ++j) tmem_ld32_start(t_s + 32 * j, s[j]);
        if (i + 1 == turns && lane == 0) mbar_arrive(bar(c->query_free[w]));
        const uint32_t *known = c->mask[which & (kMasks - 1)];
        const uint4 fine = *reinterpret_cast<const uint4 *>(known);
        bool partly = k0 < lo || k0 + BN > hi || (fine.x & fine.y) != ~0u;
        if (BN > 64) partly |= (fine.z & fine.w) != ~0u;
        const bool masks = __any_sync(kFull, partly);
        // Before the accumulators or the weights' columns are written the last tile's
        // products must be done.  (Where the weights take the scores' place, these told.)
        bool spent = !M::kAhead || i == 0;
        // Half of the keys at a time, one copy of the code (unrolled, two thirds of the
        // stalls were for instructions).
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int j = 0; j < kHalf; ++j) tmem_ld32_end(s[j]);
          if (M::kAhead && half == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(c->taken[w]));
          }
          if (unlikely(masks)) {
#pragma unroll
            for (int j = 0; j < kHalf; ++j) {
              const int first = k0 + half * (BN / 2) + 32 * j;
              const int a = min(max(lo - first, 0), 32);
              const int z = min(max(hi - first, 0), 32);
              const uint32_t seen = (z == 32 ? ~0u : (1u << z) - 1u) & (a == 32 ? 0u : ~0u << a) &
                                    known[half * kHalf + j];
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((seen >> e) & 1)) s[j][e] = 0xff800000u;    // -inf
            }
          }
          float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
          for (int j = 0; j < kHalf; ++j)
#pragma unroll
            for (int e = 0; e < 32; e += 8)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                mx[q] = max3(mx[q], __uint_as_float(s[j][e + 2 * q]), __uint_as_float(s[j][e + 2 * q + 1]));
          const float mn = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * scale;
          top = fmaxf(top, mn);
          const bool grown = mn > m + kLazy;
          if (unlikely(__any_sync(kFull, grown))) {
            const float f = !grown ? 1.f : m == -CUDART_INF_F ? 0.f : ex2(m - mn);
            if (grown) m = mn;
            l *= f;
            if (i > 0 || half == 1) {
              // (In the second half the first one's products have been added already.)
              if (half == 1) ok = wait(ctl, bar(c->half[w]), tiles & 1);
              else if (!spent) ok = spent = wait(ctl, bar(c->spent[w]), (tiles - 1) & 1);
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t o[32];
                tmem_ld32(t_o + c0, o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(t_o + c0, o);
              }
            }
          }
          if (!spent) {
            if (!(ok = spent = wait(ctl, bar(c->spent[w]), (tiles - 1) & 1))) break;
            tc_fence_after();
          }
          const float shift = kBias - (m == -CUDART_INF_F ? 0.f : m);
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < kHalf; ++j) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float x[4];
              fma2(x[0], x[1], __uint_as_float(s[j][e]), __uint_as_float(s[j][e + 1]), scale, scale, shift, shift);
              fma2(x[2], x[3], __uint_as_float(s[j][e + 2]), __uint_as_float(s[j][e + 3]), scale, scale, shift,
                   shift);
#pragma unroll
              for (int q = 0; q < 4; ++q) x[q] = ex2(x[q]);
              pk[e / 2] = pack2<T>(x[0], x[1]);
              pk[e / 2 + 1] = pack2<T>(x[2], x[3]);
              add2(sum[0], sum[1], x[0], x[1]);
              add2(sum[2], sum[3], x[2], x[3]);
            }
            tmem_st16(t_p + half * (BN / 4) + 16 * j, pk);
          }
          if (half == 0) {
#pragma unroll
            for (int j = 0; j < kHalf; ++j) tmem_ld32_start(t_s + BN / 2 + 32 * j, s[j]);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(c->weights[w][half]));   // their products may begin
        }
        if (!ok) break;
      }
      if (!ok) break;
      if (turns > 0) {      // the last products with V
        if (!wait(ctl, bar(c->spent[w]), (tiles - 1) & 1)) break;
        tc_fence_after();
      }
      // A block that the halves share: the second hands over its sums, the first adds
      // its accumulators, in TMEM in the same lanes.
      float f_own = 1.f, f_other = 0.f;
      const bool shares = !both && it.steps > 1;
      if (shares) {
        if (w == 1) {
          c->part[0][row] = m;
          c->part[1][row] = l;
          c->part[2][row] = top;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(c->done));
          if (!wait(ctl, bar(c->read), shared_at & 1)) break;
          ++shared_at;
          release();
          continue;
        }
        if (!wait(ctl, bar(c->done), shared_at & 1)) break;
        ++shared_at;
        tc_fence_after();
        const float m2 = c->part[0][row], l2 = c->part[1][row];
        const float mm = fmaxf(m, m2), ref = mm == -CUDART_INF_F ? 0.f : mm;
        f_own = ex2(m - ref);
        f_other = ex2(m2 - ref);
        l = l * f_own + l2 * f_other;
        m = mm;
        top = fmaxf(top, c->part[2][row]);
      } else if (!both && w == 1) {
        release();
        continue;
      }
      const int packed = it.row0 + in_block, t = packed / p.group, n = it.h * p.group + packed - t * p.group;
      const bool whole = it.slot < 0;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const float f = whole ? inv : 1.f;
      f_own *= f;
      f_other *= f;
      const uint32_t t_o2 = tmem + lanes + M::o_col(1);
      float *part = whole ? nullptr : part_of<kBR>(p, blockIdx.x, it.slot) + in_block;
      float bad[4] = {0.f, 0.f, 0.f, 0.f};
      // Rows go out two lanes to a row: lanes 2 m and 2 m + 1 trade 16-byte pieces, so that a
      // store writes 32 bytes of 16 rows each, not 16 of 32.
      const int64_t at = mine ? (it.r.start + t) * p.y_stride + int64_t(n) * D : -1;
      T *out[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int64_t theirs = __shfl_sync(kFull, at, (lane & ~1) + k);
        out[k] = theirs < 0 ? nullptr : static_cast<T *>(p.y) + theirs + (lane & 1) * 8;
      }
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t o[32];
        float x[32];
        if (turns > 0) {
          tmem_ld32(t_o + c0, o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2)
          mul2(x[e], x[e + 1], __uint_as_float(o[e]), __uint_as_float(o[e + 1]), f_own, f_own);
        if (shares) {
          tmem_ld32(t_o2 + c0, o);
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            fma2(x[e], x[e + 1], __uint_as_float(o[e]), __uint_as_float(o[e + 1]), f_other, f_other, x[e], x[e + 1]);
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2)
          fma2(bad[e & 2], bad[(e & 2) + 1], x[e], x[e + 1], 0.f, 0.f, bad[e & 2], bad[(e & 2) + 1]);
        if (unlikely(!whole)) {
          if (mine) {
#pragma unroll
            for (int e = 0; e < 32; ++e) part[(c0 + e) * kBR] = x[e];
          }
        } else if (p.y_chunks) {
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            uint4 v[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float *xq = x + 8 * (k + q);
              v[q] = make_uint4(pack2<T>(xq[0], xq[1]), pack2<T>(xq[2], xq[3]), pack2<T>(xq[4], xq[5]),
                                pack2<T>(xq[6], xq[7]));
            }
            const bool upper = lane & 1;
            const uint4 got = trade(upper ? v[0] : v[1]);
            if (upper) v[0] = got;
            else v[1] = got;
#pragma unroll
            for (int q = 0; q < 2; ++q)
              if (out[q] != nullptr) *reinterpret_cast<uint4 *>(out[q] + c0 + 8 * k) = v[q];
          }
        } else if (mine) {
          T *y = static_cast<T *>(p.y) + at + c0;
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = from_f<T>(x[e]);
        }
      }
      if (shares) {         // the second half may go on
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(c->read));
      }
      const uint32_t bads = __ballot_sync(kFull, mine && whole && !(bad[0] + bad[1] + bad[2] + bad[3] == 0.f));
      if (it.first) {
        uint32_t *flags = p.flags + int64_t(it.item) * (kBR / 32);
        if (lane == 0) {
          if (bads) c->flagged = 1;
          flags[(both ? w * 4 : 0) + quarter] = bads;
          if (!both) flags[4 + quarter] = 0;
        }
      }
      if (mine) {
        if (whole) {
          const float shift = (m == -CUDART_INF_F ? 0.f : m - top) - kBias;
          write_stats(p, int64_t(it.r.start + t) * p.n + n, top * kLn2, l * ex2(shift));
        } else {
          part[D * kBR] = m;
          part[(D + 1) * kBR] = l;
          part[(D + 2) * kBR] = top;
        }
      }
      tc_fence_before();    // the accumulators have been read
      release();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (tid == 0) {
    c->record.flagged = c->flagged;
    c->record.odd = c->odd;
    reinterpret_cast<Record *>(p.records)[blockIdx.x] = c->record;
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

EncodeFn extend_encode_fn() {
  static const EncodeFn fn = [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<EncodeFn>(ptr);
  }();
  return fn;
}

// The cache as a 4-D tensor, copied in boxes of `box` keys and 64 columns.  box stays 0
// where a copy would have fewer than 4 keys, more than a warp's lanes for a tile, or the
// strides are not those of nested axes, as TMA wants them.  (The swizzle goes by the
// shared memory's address, so that 4 rows are half of an atom.)
template <typename T, int D>
void make_page_maps(ExtendMaps &maps, const ExtendParams &p) {
  maps.box = 0;
  int keys = Dim<D>::BN;
  while (keys >= 4 && p.page_size % keys != 0) keys >>= 1;
  const EncodeFn enc = extend_encode_fn();
  if (enc == nullptr || keys < 4) return;
  const int64_t count[3] = {p.n_kv, p.page_size, p.num_pages};
  const int64_t stride[3] = {p.head_stride, p.token_stride, p.page_stride};
  cuuint64_t dims[4] = {D}, strides[3];
  cuuint32_t box[4] = {64, 1, 1, 1};
  const auto nested = [&](bool token_first) {
    const int order[3] = {token_first ? 1 : 0, token_first ? 0 : 1, 2};
    int64_t inner = 1, extent = D;   // stride and extent of the axis before, in elements
    for (int i = 0; i < 3; ++i) {
      const int a = order[i];
      const int64_t own = count[a] == 1 ? extent : stride[a];   // (an axis of one: any will do)
      if (own < extent || own % inner != 0 || own * int64_t(sizeof(T)) % 16 != 0 ||
          own * int64_t(sizeof(T)) >= (int64_t(1) << 40))
        return false;
      inner = own;
      extent = own * count[a];
      dims[i + 1] = cuuint64_t(count[a]);
      strides[i] = cuuint64_t(own) * sizeof(T);
      box[i + 1] = a == 1 ? cuuint32_t(keys) : 1;
    }
    maps.token_first = token_first;
    return true;
  };
  if (!nested(false) && !nested(true)) return;
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  const CUtensorMapDataType type = std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                  : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto encode = [&](CUtensorMap *map, const void *base) {
    return enc(map, type, 4, const_cast<void *>(base), dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (encode(&maps.k, p.kc) && encode(&maps.v, p.vc)) maps.box = keys;
}

// The query rows as [tokens][heads][D], copied in boxes of 128 packed rows.
template <typename T>
void make_query_map(ExtendMaps &maps, const ExtendParams &p) {
  const EncodeFn enc = extend_encode_fn();
  maps.by_tma = 0;
  if (enc == nullptr || !p.q_chunks || p.sign != 1 || 128 % p.group != 0 || p.q_stride >= (int64_t(1) << 38))
    return;
  const cuuint64_t dims[3] = {cuuint64_t(p.d), cuuint64_t(p.n), cuuint64_t(p.tokens)};
  const cuuint64_t strides[2] = {cuuint64_t(p.d) * sizeof(T), cuuint64_t(p.q_stride) * sizeof(T)};
  const cuuint32_t box[3] = {64, cuuint32_t(p.group), cuuint32_t(128 / p.group)};
  const cuuint32_t ones[3] = {1, 1, 1};
  maps.by_tma = enc(&maps.q, std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                            : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                    3, const_cast<void *>(p.q), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
cudaError_t launch_dim(const ExtendParams &p, int ctas, cudaStream_t s) {
  using M = Dim<D>;
  ExtendMaps maps{};
  make_page_maps<T, D>(maps, p);
  make_query_map<T>(maps, p);
  cudaError_t e = cudaFuncSetAttribute(extend_tc_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       M::kSmem);
  if (e != cudaSuccess) return e;
  extend_tc_kernel<T, D><<<ctas, kThreads, M::kSmem, s>>>(p, maps);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_join<T, D, kBR, M::BN>(p, ctas, s);
}

}  // namespace
}  // namespace fav
