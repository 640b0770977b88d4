// Attention of the nodes of drafted trees over a paged key-value cache.
//
//   out[t,h] = sum_j p_j V_j / sum_j p_j,   p_j = exp(scale q[t,h] . K_j)
//
// over a request's cached tokens and the nodes of t's mask. All nodes of a request read the same keys, and G = q_heads /
// kv_heads query heads share a key-value head: n G rows use each cached byte, 2 n G flops a 16-bit element. At 8 nodes and
// 6 heads that is 48 rows, which mma.sync could just feed; at 26 nodes it could not, so the products run on tcgen05, with 128 rows
// (node, head) to a tile: S = Q K^T and O += P V with S, P and O in tensor memory.
//
// Work. A (request, key-value head, 128 rows) is a segment; its keys are cut into tiles of 64. Where the segments are few and short,
// each goes to a cluster of blocks that join their parts through shared memory (kCluster). Else the tiles of all segments form
// one list, cut into equal shares for the blocks of one resident wave, so that ragged lengths need no plan from the
// host (kList): a segment inside one block's share is finished there; one that is cut leaves partial (m, l, o) in the workspace, and
// a second small kernel joins them, in block order.
//
// Warps. Four (a thread to a row) turn S into P and write results; one issues the MMAs; three or four load keys and values. Tiles go through a
// ring of slots in the order in which the MMAs take them: K0, K1, V0, K2, V1, ... All of a block's MMAs come from one thread and
// so run in order, which is what lets S of tile i + 2 overwrite P of tile i without a wait.
//
// Softmax. One pass with a running maximum m, sum l and output o; o is rescaled only where m grows by more than 2^8 (bf16) or
// 2^3 (f16): p just has to stay in range. Probabilities enter the second product as two 16-bit parts (16 bits for bf16, 22
// for f16): one part would add an error as large as the output's own rounding.
//
// Masks. A key that only some rows see meets the others with p = 0, and 0 V is NaN where V is not finite. So in tiles that not
// every row sees whole (the nodes, the edge of a window) such values are taken out when they are loaded, and added
// at the end to the rows that see them. In the others a weight that underflowed makes an infinity NaN: a NaN channel at the end is looked into.
//
// Measured (GB300; 24 heads on 4 of 256 channels and bf16 where nothing else is said, page tables as wide as the longest request needs): one request of 577 tokens, 8 nodes 11.5 us, a
// chain of latencies (length, page, tile, two products and a softmax, cluster, output); 24 requests of 40 to 9000 tokens and 4 to 26 nodes 54
// (bytes: 28), tensor pipe 38 % busy: a tile is 2250 cycles of product, softmax, product and the waits between them, and a piece of a
// segment costs 6 us besides (queries, list, output); 64 nodes on 80001 tokens 146 (flops: 66, 100 with both parts of P), tensor pipe 65 %;
// 160 requests of 512 to 16384 tokens in 8 bits under a window of 8192, 40 heads on 8 of 128 channels 438 (bytes: 193), tensor pipe 48 %:
// of a block's 3100 cycles a tile the softmax takes 2700, on two warps (60 rows at most) beside three that widen.
#pragma once

#include <climits>

#include "paged_attention.cuh"
#include "tree.cuh"

namespace tl {

struct TreeAttnParams {
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  int64_t page_stride, head_stride, token_stride;     // bytes
  int num_pages;
  FastDiv page, group_div;
  const uint16_t* q;
  uint16_t* out;
  int64_t ldq, ldo;
  const int64_t* masks;
  const int32_t* starts;
  const int32_t* lens;
  const int32_t* pages;
  int64_t ldp;
  float* lse;
  float scale_log2;
  int B, T, q_heads, kv_heads, group, window, sinks, q_bf16, capacity;
  int runs16;                                         // page_size is a multiple of 16: 16 keys from a multiple of 16 lie at equal distances
  int cluster_log, row_blocks;                        // kCluster: 2^cluster_log blocks to a segment; row blocks that a request may have
  int grid;                                           // kList: blocks of the first kernel
  float* partials;                                    // two per block
  struct TreeCut* cuts;                               // one per block
  int* status;
};

// A segment that is cut, noted by the block in whose share it begins; parts = 0: none.
struct TreeCut {
  int parts, row0, kvh, first_row, rows;              // row0: the request's first node; first_row: of its rows (node, head)
  float v_scale;
};

constexpr int kTreeRows = 128;
constexpr int kTreeMaxGrid = 2048;

__host__ __device__ constexpr size_t tree_partial_floats(int dim) { return static_cast<size_t>(kTreeRows) * (dim + 2); }

cudaError_t launch_tree_attn_bf16(TreeAttnParams p, int dim, int sms, cudaStream_t st);
cudaError_t launch_tree_attn_f16(TreeAttnParams p, int dim, int sms, cudaStream_t st);
cudaError_t launch_tree_attn_f8(TreeAttnParams p, int dim, int sms, cudaStream_t st);

// Blocks of the first kernel on an SM, by head_dim: tensor memory and shared memory for two up to 128 channels.
__host__ __device__ constexpr int tree_blocks_per_sm(int dim) { return dim == 256 ? 1 : 2; }

namespace tree {

using attn::cp_async16;
using attn::cp_async_commit;
using attn::cp_async_wait;
using attn::exp2_approx;
using attn::faded;
using attn::pack2;
using attn::unpack2;
using attn::widen_hi;
using attn::widen_lo;

constexpr int kKeys = 64;                // keys of a tile
constexpr int kSoftmaxWarps = 4, kMmaWarp = 4, kLoadWarp = 5;
constexpr int kMaxClusterLog = 4;
// Bytes of K and V that several row blocks read, from which on they do so together, if that leaves no more than an eighth of the places empty.
// One request, 64 nodes, together and not: 20000 tokens 52.2 and 55.5 us, 40000 80.8 and 96.4, 80001 137 and 166; below, eight of 1000 tokens
// 45 and 39, 24 of 40 to 9000 62 and 59. Eight of 4000, where padding would add half: 96 and 77.
constexpr long long kReread = 64 << 20;

enum Mode {
  kList,      // the list of tiles, in equal shares, and a second kernel for the segments that are cut
  kCluster    // a cluster of blocks takes a segment, and joins it through its shared memory
};
constexpr int kAhead = 16;               // pieces: more than the loading warps can be ahead of the others, or of each other

template <int CACHE, int D>
struct Traits {
  static constexpr bool F8 = CACHE == kCacheF8, BF16 = CACHE == kCacheBf16;
  static constexpr int ROW = D * (F8 ? 1 : 2);                   // bytes of a cached row
  static constexpr int BLOCKS = tree_blocks_per_sm(D);
  // Up to eight warps are four to a scheduler for two blocks, and have 128 registers.
  static constexpr int LOADERS = BLOCKS == 1 ? 4 : 3;
  static constexpr int THREADS = 32 * (kLoadWarp + LOADERS);
  // queries as the MMA's operand in tensor memory, or, where that has no room for two buffers of S beside them, in shared memory
  static constexpr bool QT = D != 128;
  static constexpr int Q = QT ? kSoftmaxWarps * 4096 : kTreeRows * D * 2;        // the results pass through it, 4 KB a warp
  static constexpr int SLOT = kKeys * D * 2, STAGE = F8 ? SLOT / 2 : 0;
  // (slots, us: 64 channels 8 or 12: 123 or 132 of 64 requests, 128 channels 4 or 5: 99 or 101 of 40, 256 channels 6 or 4: 73 or 76 of 24)
  static constexpr int SLOTS = D == 64 ? 8 : D == 128 ? (F8 ? 3 : 4) : F8 ? 4 : 6;
  static constexpr int STAGES = F8 ? LOADERS : 0;                // of 8-bit rows on their way, a loading warp's each
  static constexpr int PART = kTreeRows * (D + 2) * 4;           // of a cluster's block, in the ring's place
  static constexpr int OFF_SLOT = Q, OFF_STAGE = OFF_SLOT + SLOTS * SLOT, END = OFF_STAGE + STAGES * STAGE;
  static constexpr int OFF_MISC = END > OFF_SLOT + PART ? END : OFF_SLOT + PART;
  static constexpr int SMEM = OFF_MISC + 1024;
  static constexpr int SBUF = 2;                                 // buffers of S and P
  static constexpr int TMEM = D == 256 ? 512 : 256, TMEM_S = D, TMEM_Q = TMEM_S + SBUF * kKeys;      // columns; O in the first D
  // What a segment costs besides its tiles (queries, results, the list: some 6 us), in tiles. Against 5 and 8 in turn: 24 requests, 256
  // channels 58.7 and 54.8 us; 60 requests, 8 bits, 235 and 218; 40 requests, 128 channels 91 and 87, in 8 bits 448 and 454; 64 channels 160 and 165.
  static constexpr int COST = D == 64 || (D == 128 && F8) ? 5 : 8;
  static constexpr float POFF = BF16 ? 0.f : 12.f;               // p is kept 2^POFF as large (f16: away from the subnormals)
  static constexpr float SLACK = BF16 ? 8.f : 3.f;               // by how much m may lag behind the maximum
  static_assert(SMEM <= (BLOCKS == 1 ? 232448 : 115712) && TMEM_Q + (QT ? D / 2 : 0) <= TMEM, "room");
  // a piece takes two slots at least, and a loading warp has one load of any LOADERS
  static_assert(SLOTS / 2 + 3 < kAhead && LOADERS <= 4, "ahead");
};

// The small things behind the slots.
template <class T>
struct Misc {
  uint64_t full[T::SLOTS], empty[T::SLOTS];            // a slot holds its rows; its MMAs are done
  uint64_t s_full[T::SBUF], p_full[T::SBUF], pv_done[T::SBUF];
  uint64_t q_full;                                     // a piece's queries are in place
  uint64_t loaded[kAhead];                             // a piece's last rows are, and flag says what was found in them
  int flag[kAhead];                                    // piece + 1 where values were taken out
  int bad[kAhead];                                     // 0, or of the keys whose page does not exist the last one, plus 1
  uint32_t tmem;
  int abort;
};

// ---- PTX
// MMAs in straight-line blocks, with 32-bit arithmetic on the descriptors (all of which have the same upper half): a thread that builds
// every descriptor anew issues an MMA in 82 cycles, which is longer than one of 64 columns takes.
// S (+)= Q K^T for 64 channels, Q in tensor memory (8 columns for 16 channels)
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t bhi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p0, p1;\n .reg .b64 bd;\n .reg .b32 t;\n"
      "setp.ne.b32 p0, %5, 0;\n setp.eq.b32 p1, %2, %2;\n"
      "mov.b64 bd, {%2, %3};\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], bd, %4, p0;\n"
      "add.u32 t, %2, 2;\n mov.b64 bd, {t, %3};\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1+8], bd, %4, p1;\n"
      "add.u32 t, %2, 4;\n mov.b64 bd, {t, %3};\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1+16], bd, %4, p1;\n"
      "add.u32 t, %2, 6;\n mov.b64 bd, {t, %3};\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1+24], bd, %4, p1;\n"
      "}" ::"r"(d), "r"(a), "r"(b), "r"(bhi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// the same with Q in shared memory
__device__ __forceinline__ void mma4_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p0, p1;\n .reg .b64 ad, bd;\n .reg .b32 t;\n"
      "setp.ne.b32 p0, %5, 0;\n setp.eq.b32 p1, %2, %2;\n"
      "mov.b64 ad, {%1, %3};\n mov.b64 bd, {%2, %3};\n tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %4, p0;\n"
      "add.u32 t, %1, 2;\n mov.b64 ad, {t, %3};\n add.u32 t, %2, 2;\n mov.b64 bd, {t, %3};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %4, p1;\n"
      "add.u32 t, %1, 4;\n mov.b64 ad, {t, %3};\n add.u32 t, %2, 4;\n mov.b64 bd, {t, %3};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %4, p1;\n"
      "add.u32 t, %1, 6;\n mov.b64 ad, {t, %3};\n add.u32 t, %2, 6;\n mov.b64 bd, {t, %3};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %4, p1;\n"
      "}" ::"r"(d), "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// O (+)= P V for 64 keys: for each 16 of them 8 columns of high parts, 8 of low ones, and 2048 bytes of V
__device__ __forceinline__ void mma8_pv(uint32_t d, uint32_t a, uint32_t b, uint32_t bhi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p0, p1;\n .reg .b64 bd;\n .reg .b32 t;\n"
      "setp.ne.b32 p0, %5, 0;\n setp.eq.b32 p1, %2, %2;\n"
      "mov.b64 bd, {%2, %3};\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], bd, %4, p0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1+8], bd, %4, p1;\n"
      "add.u32 t, %2, 128;\n mov.b64 bd, {t, %3};\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1+16], bd, %4, p1;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1+24], bd, %4, p1;\n"
      "add.u32 t, %2, 256;\n mov.b64 bd, {t, %3};\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1+32], bd, %4, p1;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1+40], bd, %4, p1;\n"
      "add.u32 t, %2, 384;\n mov.b64 bd, {t, %3};\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1+48], bd, %4, p1;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1+56], bd, %4, p1;\n"
      "}" ::"r"(d), "r"(a), "r"(b), "r"(bhi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Both barriers see one arrival when the MMAs issued so far are done.
__device__ __forceinline__ void commit2(uint32_t bar1, uint32_t bar2) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n"
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];" ::"r"(bar1),
      "r"(bar2)
      : "memory");
}
// A 64-channel column block of 128-byte rows, 128-byte swizzle; the operand's other dimension is along the rows (K-major: next 8
// rows at 1024 bytes), or the summed one is (MN-major: next 8 rows at 1024 bytes, the next 64 channels at `block` bytes).
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t block) {
  uint64_t d = smem_desc_sw128(saddr);
  d &= ~(static_cast<uint64_t>(0x3FFF) << 16);
  return d | static_cast<uint64_t>(block >> 4) << 16;
}
template <bool BF16>
__host__ __device__ constexpr uint32_t idesc(int n, bool b_mn_major) {
  return idesc_f16_f32(kTreeRows, n) | (BF16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn_major ? 1u << 16 : 0u);
}

// byte offset of 16-byte unit u (of 8) of row r in a 64-channel block
__device__ __forceinline__ uint32_t swizzled(int r, int u) { return r * 128 + ((u ^ (r & 7)) << 4); }

// bits 0 .. n - 1
__device__ __forceinline__ uint64_t low_bits(int n) { return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1; }

// All lanes of a warp wait for a phase, and know alike whether it came.
__device__ __forceinline__ bool wait_all(uint64_t& bar, uint32_t parity, int* abort, int* status) {
  const bool ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar), parity & 1, abort));
  if (!ok) {
    set_status(status, TL_ETIMEOUT);
    *const_cast<volatile int*>(abort) = 1;
  }
  return ok;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Waits for the loads from tensor memory so far (the registers pass through the wait, so that no use of them comes before it).
__device__ __forceinline__ void arrived(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]),
                 "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]),
                 "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]),
                 "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])::"memory");
}

// 32 columns of this warp's lanes, there when it returns.
__device__ __forceinline__ void read_tmem(uint32_t addr, uint32_t (&v)[32]) {
  tmem_ld_32x32b_x32(addr, v);
  arrived(v);
}

// ---- the list of work: every warp goes through its block's share by itself
struct Request {
  int n, row0, len, first, begin, sinks, sink_tiles, tiles, row_blocks;
  __device__ __forceinline__ int places(int cost) const { return row_blocks == 0 ? 0 : tiles + cost; }
};

__device__ __forceinline__ Request request(const TreeAttnParams& p, int b, bool& bad) {
  Request r;
  const bool ok = tree_rows(p.starts, b, p.T, r.row0, r.n);
  r.len = __ldg(p.lens + b);
  if (!ok || r.len < 0 || r.len > p.capacity - r.n) {
    bad = true;
    r.n = r.len = 0;
  }
  r.first = p.window > 0 ? max(0, r.len - p.window) : 0;      // the first key that any row's window reaches
  r.begin = p.runs16 ? r.first & ~15 : r.first;               // its tiles begin with that key's run
  r.sinks = min(p.sinks, r.first);
  r.sink_tiles = (r.sinks + kKeys - 1) / kKeys;
  r.tiles = r.sink_tiles + (r.len + r.n - r.begin + kKeys - 1) / kKeys;
  r.row_blocks = (r.n * p.group + kTreeRows - 1) / kTreeRows;
  return r;
}

struct Piece {              // tiles begin .. end - 1 of a segment
  int kvh, row_block, begin, end;
  bool whole, starts_here;
  int second, parts;        // which of the block's partials; blocks that share the segment
};

template <Mode MODE, int COST>
struct Walk {
  Request r;
  int b, seg, segs;         // request, segment of it, its segments
  int places;               // of a segment of this request
  long long at, share, t1;  // place where the segment begins; places of a share; where this block's share ends
  long long t0;
  bool more;

  // Where several row blocks share many keys, each one's places are a whole number of shares: then the blocks that read the same
  // keys do so at the same time, and all but the first find them in L2.
  __device__ __forceinline__ int padded(int n, int row_blocks, bool together) const {
    if (!together || row_blocks < 2 || n <= share) return n;
    const int s = static_cast<int>(share);
    return (n + s - 1) / s * s;
  }

  // All lanes of a warp together. `tile_bytes`: of K and V of a tile.
  __device__ __forceinline__ void init(const TreeAttnParams& p, int tile_bytes, bool report) {
    const int lane = threadIdx.x & 31;
    bool bad = false;
    if constexpr (MODE == kCluster) {
      b = static_cast<int>((blockIdx.x >> p.cluster_log) / static_cast<unsigned>(p.kv_heads * p.row_blocks));
      seg = static_cast<int>(blockIdx.x >> p.cluster_log) - b * p.kv_heads * p.row_blocks;
      r = request(p, b, bad);
      if (report && bad && lane == 0) set_status(p.status, TL_EDATA);
      more = seg % p.row_blocks < r.row_blocks;
      return;
    }
    // what a lane knows of its request, of up to 32 for good
    int n = 0, row_blocks = 0;
    auto look = [&](int base) {
      n = row_blocks = 0;
      if (base + lane >= p.B) return;
      const Request x = request(p, base + lane, bad);
      n = x.places(COST), row_blocks = x.row_blocks;
    };
    look(0);
    share = 0;
    bool together = false;
    long long total, again = 0, apart = 0, bare = 0;  // apart, bare: share and total without padding
    for (;;) {              // the least share with which the places fit the blocks, within 3 %
      total = 0;
      for (int base = 0; base < p.B; base += 32) {
        if (p.B > 32) look(base);
        total += static_cast<long long>(p.kv_heads) * row_blocks * padded(n, row_blocks, together);
        if (share == 0 && row_blocks > 1) again += static_cast<long long>(p.kv_heads) * n * tile_bytes;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      const long long least = attn::divide(total + p.grid - 1, p.grid);
      if (least <= share) break;
      if (share == 0) {
        share = apart = least, bare = total;
        if (!__any_sync(0xffffffffu, row_blocks > 1 || again > 0)) break;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) again += __shfl_xor_sync(0xffffffffu, again, o);
        together = again > kReread && share < (1 << 30);
        if (!together) break;
      } else {
        share = max(least, share + share / 32);
        if (share > apart + apart / 8) {                // too much would stay empty
          together = false, share = apart, total = bare;
          break;
        }
      }
    }
    if (report && bad) set_status(p.status, TL_EDATA);
    t0 = share * blockIdx.x;
    t1 = min(t0 + share, total);
    more = t0 < total;
    if (!more) return;
    long long run = 0;
    for (int base = 0;; base += 32) {
      if (base >= p.B) {                                // (lengths that change meanwhile: nothing is looked up past the last request)
        more = false;
        return;
      }
      if (p.B > 32) look(base);
      const long long mine = static_cast<long long>(p.kv_heads) * row_blocks * padded(n, row_blocks, together);
      long long incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned who = __ballot_sync(0xffffffffu, t0 < run + incl);
      if (who != 0) {
        const int l = __ffs(who) - 1;
        b = base + l;
        at = run + __shfl_sync(0xffffffffu, incl - mine, l);
        break;
      }
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    join = together;
    r = request(p, b, bad);
    enter(p);
    seg = static_cast<int>(attn::divide(t0 - at, places));
    at += static_cast<long long>(seg) * places;
  }
  bool join;                // (of `padded`)

  __device__ __forceinline__ void enter(const TreeAttnParams& p) {
    places = padded(r.places(COST), r.row_blocks, join);
    segs = p.kv_heads * r.row_blocks;
    seg = 0;
  }

  // The next piece with tiles in it; false at the end of the share.
  __device__ __forceinline__ bool next(const TreeAttnParams& p, Piece& x) {
    if constexpr (MODE == kCluster) {
      if (!more) return false;
      more = false;
      const int rank = blockIdx.x & ((1 << p.cluster_log) - 1);
      x.kvh = seg / p.row_blocks;
      x.row_block = seg - x.kvh * p.row_blocks;
      x.begin = static_cast<int>(static_cast<long long>(r.tiles) * rank >> p.cluster_log);
      x.end = static_cast<int>(static_cast<long long>(r.tiles) * (rank + 1) >> p.cluster_log);
      x.whole = p.cluster_log == 0;
      x.starts_here = false, x.second = 0, x.parts = 0;
      return x.end > x.begin;
    } else {
    while (more) {
      if (at >= t1) {
        more = false;
        break;
      }
      if (seg == segs) {
        bool bad = false;
        if (b + 1 >= p.B) {
          more = false;
          break;
        }
        r = request(p, ++b, bad);
        enter(p);
        continue;
      }
      // (what is left of a whole number of shares stays empty)
      const long long from = max(t0 - at, 0ll) - COST, to = min(t1 - at, static_cast<long long>(r.places(COST))) - COST;
      x.begin = static_cast<int>(max(from, 0ll));
      x.end = static_cast<int>(max(to, 0ll));
      x.kvh = seg / r.row_blocks;
      x.row_block = seg - x.kvh * r.row_blocks;
      x.whole = x.begin == 0 && x.end == r.tiles;
      x.starts_here = x.begin == 0;
      x.second = x.starts_here;
      x.parts = 1;
      if (!x.whole && x.starts_here)
        x.parts = static_cast<int>(attn::divide(at + COST + r.tiles - 1, share)) - static_cast<int>(blockIdx.x) + 1;
      ++seg;
      at += places;
      if (x.end > x.begin) return true;
    }
    return false;
    }
  }
};

// A tile of a request: its first key, one past its last, and whether all rows see all of its 64 keys.
struct Tile {
  int k0, end;
  bool sink, plain;
};

__device__ __forceinline__ Tile tile(const TreeAttnParams& p, const Request& r, int i) {
  Tile t;
  t.sink = i < r.sink_tiles;
  t.k0 = t.sink ? i * kKeys : r.begin + (i - r.sink_tiles) * kKeys;
  t.end = min(t.k0 + kKeys, t.sink ? r.sinks : r.len + r.n);
  // a row's window holds up to TL_TREE_NODES nodes of its own and so many cached keys fewer
  t.plain = t.sink ? t.end - t.k0 == kKeys
                   : t.k0 + kKeys <= r.len && (p.window == 0 || t.k0 >= r.len - p.window + TL_TREE_NODES);
  return t;
}

// Which of a tile's keys the row with this mask sees.
__device__ __forceinline__ uint64_t visible(const TreeAttnParams& p, const Request& r, const Tile& t, uint64_t mask) {
  if (t.sink) return low_bits(t.end - t.k0);
  const int first = p.window > 0 ? max(0, r.len - max(0, p.window - __popcll(mask))) : 0;
  const int nodes = r.len - t.k0;                     // where the nodes begin
  const uint64_t cached = low_bits(nodes) & ~low_bits(r.first - t.k0) & (~low_bits(first - t.k0) | low_bits(p.sinks - t.k0));
  const uint64_t drafted = nodes >= 64 ? 0 : nodes >= 0 ? mask << nodes : nodes > -64 ? mask >> -nodes : 0;
  return cached | drafted;
}

__device__ __forceinline__ void st_shared(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// ---- the loading warps: rows of K and V into the ring's slots. They take the loads in turn, each a whole one: looking the rows' addresses up
// takes as long as copying them, and all warps together at every load took 3000 cycles for a tile of 256 channels.
template <int CACHE, int D, Mode MODE>
struct Loader {
  using T = Traits<CACHE, D>;
  static constexpr int CPR = T::ROW / 16;               // 16-byte chunks of a cached row
  static constexpr int RPI = 32 / CPR;                  // rows that one instruction copies
  static constexpr int STEPS = kKeys / RPI;

  const TreeAttnParams& p;
  uint8_t* smem;
  Misc<T>* misc;
  int warp, lane;                                       // of the loading warps
  int pieces = 0;                                       // whose loads are done
  bool ok = true;

  // Where a tile's rows lie. With runs of 16, lanes 0 to 3 know the first row of theirs; otherwise a lane the rows of keys lane and lane + 32.
  struct Rows {
    int64_t off[2];                                     // byte offset in the cache, or -1
  };
  __device__ __forceinline__ void pages_of(const int32_t* pages, const Tile& t, int (&page)[2]) const {
    const int key = t.k0 + (p.runs16 ? 16 * (lane & 3) : lane);
    page[0] = key < t.end ? __ldg(pages + p.page.div(key)) : -1;
    page[1] = !p.runs16 && key + 32 < t.end ? __ldg(pages + p.page.div(key + 32)) : -1;
  }
  __device__ __forceinline__ int64_t row_of(int key, int page, const Tile& t, int64_t head) const {
    if (key >= t.end) return -1;
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) {      // (what a window leaves of it is looked into at the piece's end)
      atomicMax(&misc->bad[pieces % kAhead], key < p.sinks ? INT_MAX : key + (p.runs16 ? 16 : 1));
      return -1;
    }
    return page * p.page_stride + head + static_cast<int64_t>(key - p.page.div(key) * p.page.d) * p.token_stride;
  }
  __device__ __forceinline__ void rows_of(const Tile& t, const int (&page)[2], int64_t head, Rows& r) const {
    const int key = t.k0 + (p.runs16 ? 16 * (lane & 3) : lane);
    r.off[0] = row_of(key, page[0], t, head);
    r.off[1] = p.runs16 ? -1 : row_of(key + 32, page[1], t, head);
  }

  // A lane copies chunk lane % CPR of rows lane / CPR, + RPI, ...; dst(i): where that of instruction i goes. Rows that are not there become zeros.
  template <typename F>
  __device__ __forceinline__ void copy(const uint8_t* base, const Rows& rows, const Tile& t, F&& dst) const {
    const int row = lane / CPR;
    base += lane % CPR * 16;
    if (p.runs16) {
      constexpr int G = 16 / RPI;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int64_t o = __shfl_sync(0xffffffffu, rows.off[0], g);
        const int left = o < 0 ? 0 : t.end - t.k0 - 16 * g - row;      // rows of this lane on
        const uint8_t* from = base + (o < 0 ? 0 : o) + row * p.token_stride;
#pragma unroll
        for (int i = 0; i < G; ++i) {
          cp_async16(dst(g * G + i), left > i * RPI ? from : base, left > i * RPI ? 16u : 0u);
          from += RPI * p.token_stride;
        }
      }
    } else {
#pragma unroll 2
      for (int i = 0; i < STEPS; ++i) {
        const int64_t o = __shfl_sync(0xffffffffu, i * RPI < 32 ? rows.off[0] : rows.off[1], (i * RPI + row) & 31);
        cp_async16(dst(i), base + (o < 0 ? 0 : o), o < 0 ? 0u : 16u);
      }
    }
  }

  // For load i: load i - SLOTS has been taken. A wait tells a phase from its neighbours only where the one before is known to be
  // over: this warp's last wait said so of all loads up to i - LOADERS - SLOTS, and load i - 2 SLOTS has to be among them.
  __device__ __forceinline__ void wait_empty(uint32_t i) {
    static_assert(T::LOADERS <= T::SLOTS, "phases");
    if (i >= T::SLOTS) ok = wait_all(misc->empty[i % T::SLOTS], i / T::SLOTS - 1, &misc->abort, p.status);
  }
  __device__ __forceinline__ void note_odd() const { *const_cast<volatile int*>(&misc->flag[pieces % kAhead]) = pieces + 1; }

  // 16 bits: straight into slot n % SLOTS; the copies themselves arrive when they have landed.
  __device__ __forceinline__ void load16(uint32_t n, const uint8_t* base, const Rows& rows, const Tile& t, bool check) {
    wait_empty(n);
    if (!ok) return;
    const int row = lane / CPR, chunk = lane % CPR, off = T::OFF_SLOT + n % T::SLOTS * T::SLOT + chunk / 8 * (kKeys * 128);
    copy(base, rows, t, [&](int i) { return smem_u32(smem) + off + swizzled(i * RPI + row, chunk % 8); });
    const uint32_t full = smem_u32(&misc->full[n % T::SLOTS]);
    if (!check) {
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full) : "memory");
      return;
    }
    cp_async_commit();
    cp_async_wait<0>();
    // an exponent of ones, plus one in its last place, carries into the sign's place
    constexpr uint32_t E = T::BF16 ? 0x7F807F80u : 0x7C007C00u, ONE = T::BF16 ? 0x00800080u : 0x04000400u;
    uint32_t any = 0;
#pragma unroll 8
    for (int i = 0; i < STEPS; ++i) {
      const uint4 x = *reinterpret_cast<const uint4*>(smem + off + swizzled(i * RPI + row, chunk % 8));
      any |= ((x.x & E) + ONE) | ((x.y & E) + ONE) | ((x.z & E) + ONE) | ((x.w & E) + ONE);
    }
    if ((any & 0x80008000u) != 0) {
      note_odd();
#pragma unroll 1
      for (int i = 0; i < STEPS; ++i) {
        uint4* const at = reinterpret_cast<uint4*>(smem + off + swizzled(i * RPI + row, chunk % 8));
        const uint4 x = *at;
        *at = make_uint4(x.x & ~__vcmpeq2(x.x & E, E), x.y & ~__vcmpeq2(x.y & E, E), x.z & ~__vcmpeq2(x.z & E, E), x.w & ~__vcmpeq2(x.w & E, E));
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(full);
  }

  // 8 bits: into this warp's stage, and from there to the slot as f16. (While one warp widens, the others' rows are on their way.)
  __device__ __forceinline__ void load8(uint32_t n, const uint8_t* base, const Rows& rows, const Tile& t, bool check) {
    const int row = lane / CPR, chunk = lane % CPR;
    uint8_t* const stage = smem + T::OFF_STAGE + warp * T::STAGE + chunk * 16;
    copy(base, rows, t, [&](int i) { return smem_u32(stage) + (i * RPI + row) * T::ROW; });
    cp_async_commit();
    cp_async_wait<0>();
    wait_empty(n);
    if (!ok) return;
    if (check) {                                        // e4m3 has NaN (0x7F, 0xFF), no infinities
      constexpr uint32_t N = 0x7F7F7F7Fu;
      bool found = false;
#pragma unroll 1
      for (int i = 0; i < STEPS; ++i) {
        uint4* const at = reinterpret_cast<uint4*>(stage + (i * RPI + row) * T::ROW);
        const uint4 x = *at;
        const uint32_t a = __vcmpeq4(x.x & N, N), b = __vcmpeq4(x.y & N, N), c = __vcmpeq4(x.z & N, N), d = __vcmpeq4(x.w & N, N);
        if ((a | b | c | d) != 0) *at = make_uint4(x.x & ~a, x.y & ~b, x.z & ~c, x.w & ~d), found = true;
      }
      if (found) note_odd();
    }
    // Lanes of the two 64-channel blocks write their halves in different order: different banks. (All loads of a batch before its
    // conversions: one after the other took three times as long.)
    const bool turn = chunk & 4;
    const uint32_t from = smem_u32(stage) + row * T::ROW;
    const uint32_t to = smem_u32(smem) + T::OFF_SLOT + n % T::SLOTS * T::SLOT + chunk / 4 * (kKeys * 128) + row * 128 + (((chunk % 4 * 2 + turn) ^ (row & 7)) << 4);
    constexpr int BATCH = STEPS < 8 ? STEPS : 8;
#pragma unroll
    for (int i0 = 0; i0 < STEPS; i0 += BATCH) {
      uint4 x[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) x[i] = ld_shared(from + (i0 + i) * (RPI * T::ROW));
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        if (turn) x[i] = make_uint4(x[i].z, x[i].w, x[i].x, x[i].y);
        const int r = (i0 + i) * RPI;
        const uint32_t at = (to ^ ((r & 7) << 4)) + r * 128;
        st_shared(at, make_uint4(widen_lo(x[i].x), widen_hi(x[i].x), widen_lo(x[i].y), widen_hi(x[i].y)));
        st_shared(at ^ 16, make_uint4(widen_lo(x[i].z), widen_hi(x[i].z), widen_lo(x[i].w), widen_hi(x[i].w)));
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(smem_u32(&misc->full[n % T::SLOTS]));
  }

  __device__ __forceinline__ void run() {
    Walk<MODE, T::COST> w;
    w.init(p, 2 * kKeys * T::ROW, false);
    Piece x;
    uint32_t before = 0;                                // loads of the pieces before
    while (ok && w.next(p, x)) {
      // loads K0, K1, V0, K2, V1, ... of n tiles
      const int n = x.end - x.begin;
      auto tile_of = [&](int j) { return tile(p, w.r, x.begin + (j == 2 * n - 1 ? n - 1 : j & 1 ? (j + 1) / 2 : j == 0 ? 0 : j / 2 - 1)); };
      int j = (warp + T::LOADERS - static_cast<int>(before % T::LOADERS)) % T::LOADERS;
      const int32_t* const pages = p.pages + w.b * p.ldp;
      const int64_t head = x.kvh * p.head_stride;
      int page[2] = {-1, -1};
      Tile t{};
      if (j < 2 * n) {
        t = tile_of(j);
        pages_of(pages, t, page);
      }
      for (; ok && j < 2 * n; j += T::LOADERS) {
        const Tile now = t;
        Rows rows;
        rows_of(now, page, head, rows);
        if (j + T::LOADERS < 2 * n) {
          t = tile_of(j + T::LOADERS);
          pages_of(pages, t, page);
        }
        const bool v = j == 2 * n - 1 || (j != 0 && !(j & 1));
        if constexpr (T::F8)
          load8(before + j, v ? p.v : p.k, rows, now, v && !now.plain);
        else
          load16(before + j, v ? p.v : p.k, rows, now, v && !now.plain);
      }
      before += 2 * n;
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&misc->loaded[pieces % kAhead]));      // this warp's part of the piece
      ++pieces;
    }
    cp_async_wait<0>();
  }
};

// ---- the MMA warps. Loads come as K0, K1, V0, K2, V1, ... of a piece of n tiles: K_i is load max(2 i - 1, 0), V_i load min(2 i + 2, 2 n - 1).
template <int CACHE, int D, Mode MODE>
struct Mma {
  using T = Traits<CACHE, D>;
  static constexpr uint32_t ID_S = idesc<T::BF16>(kKeys, false), ID_O = idesc<T::BF16>(D, true);
  const TreeAttnParams& p;
  uint8_t* smem;
  Misc<T>* misc;
  uint32_t elected = 0, tm = 0, lo = 0, khi = 0, vlo = 0, vhi = 0;
  bool ok = true;

  __device__ __forceinline__ void init() {
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(elected));
    tm = misc->tmem;
    const uint64_t kd = smem_desc_sw128(smem_u32(smem)), vd = desc_mn(smem_u32(smem), kKeys * 128);      // of the first byte of shared memory
    lo = static_cast<uint32_t>(kd), khi = static_cast<uint32_t>(kd >> 32), vlo = static_cast<uint32_t>(vd), vhi = static_cast<uint32_t>(vd >> 32);
  }
  __device__ __forceinline__ bool wait(uint64_t& bar, uint32_t parity) { return ok = ok && wait_all(bar, parity, &misc->abort, p.status); }

  __device__ __forceinline__ bool ready(uint64_t& bar, uint32_t parity) const { return mbar_try_wait(smem_u32(&bar), parity & 1); }

  // S of tile t, K being load n, which is there. S's buffer was P's of two tiles ago: the MMAs that read it were issued before, and
  // one thread's MMAs run in order.
  __device__ __forceinline__ void scores(uint32_t t, uint32_t n) {
    const uint32_t buf = t % T::SBUF, s = n % T::SLOTS;
    if (elected) {
      const uint32_t k = lo + (T::OFF_SLOT + s * T::SLOT) / 16;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        if constexpr (T::QT)
          mma4_ts(tm + T::TMEM_S + buf * kKeys, tm + T::TMEM_Q + 32 * c, k + c * (kKeys * 128 / 16), khi, ID_S, c > 0);
        else
          mma4_ss(tm + T::TMEM_S + buf * kKeys, lo + c * (kTreeRows * 128 / 16), k + c * (kKeys * 128 / 16), khi, ID_S, c > 0);
      }
      commit2(smem_u32(&misc->empty[s]), smem_u32(&misc->s_full[buf]));
    }
    __syncwarp();
  }
  // O (+)= P V of tile t, V being load n.
  __device__ __forceinline__ void output(uint32_t t, uint32_t n, bool first) {
    const uint32_t buf = t % T::SBUF, s = n % T::SLOTS;
    if (elected) {
      mma8_pv(tm, tm + T::TMEM_S + buf * kKeys, vlo + (T::OFF_SLOT + s * T::SLOT) / 16, vhi, ID_O, !first);
      commit2(smem_u32(&misc->empty[s]), smem_u32(&misc->pv_done[buf]));
    }
    __syncwarp();
  }
  // Load n is there, for the MMAs to read what ordinary copies wrote.
  __device__ __forceinline__ bool take(uint32_t n) {
    if (!wait(misc->full[n % T::SLOTS], n / T::SLOTS)) return false;
    fence_proxy_async_smem();
    tc_fence_after();
    return true;
  }

  // S_0, S_1, O_0, S_2, O_1, ... A wait takes 200 cycles even where nothing is to be waited for, and four of them a tile left the tensor cores
  // idle for a third of the time: so the three barriers of a step are asked together.
  __device__ __forceinline__ void run() {
    init();
    Walk<MODE, T::COST> w;
    w.init(p, 2 * kKeys * T::ROW, false);
    Piece x;
    uint32_t before = 0, tiles = 0, pieces = 0;
    while (ok && w.next(p, x)) {
      const uint32_t n = x.end - x.begin;
      if (!wait(misc->q_full, pieces) || !take(before)) break;
      scores(tiles, before);
      if (n > 1) {
        if (!take(before + 1)) break;
        scores(tiles + 1, before + 1);
      }
#pragma unroll 1
      for (uint32_t i = 0; ok && i < n; ++i, ++tiles) {
        const uint32_t buf = tiles % T::SBUF, v = before + min(2 * i + 2, 2 * n - 1), k = before + 2 * i + 3;
        const bool more = i + 2 < n;
        const bool p_there = ready(misc->p_full[buf], tiles / T::SBUF), v_there = ready(misc->full[v % T::SLOTS], v / T::SLOTS);
        const bool k_there = more && ready(misc->full[k % T::SLOTS], k / T::SLOTS);
        const unsigned there = __reduce_and_sync(0xffffffffu, (p_there && v_there ? 1u : 0u) | (k_there ? 2u : 0u));
        if (!(there & 1u) && (!wait(misc->p_full[buf], tiles / T::SBUF) || !wait(misc->full[v % T::SLOTS], v / T::SLOTS))) break;
        fence_proxy_async_smem();
        tc_fence_after();
        output(tiles, v, i == 0);
        if (more) {
          if (!(there & 2u) && !take(k)) break;
          scores(tiles + 2, k);
        }
      }
      before += 2 * n;
      ++pieces;
    }
  }
};

// ---- the softmax warps: thread = row
template <int CACHE, int D, Mode MODE>
struct Softmax {
  using T = Traits<CACHE, D>;
  const TreeAttnParams& p;
  uint8_t* smem;
  Misc<T>* misc;
  int warp, lane;
  bool ok = true;

  __device__ __forceinline__ bool wait(uint64_t& bar, uint32_t parity) { return ok = ok && wait_all(bar, parity, &misc->abort, p.status); }

  // Queries and results are read and written 128 bytes of a row by eight lanes, four rows an instruction: place k of a lane is row
  // 4 k + lane / 8 of its warp. (A row to a lane made 32 lines of every instruction.) They pass through 4 KB of shared memory, 128 bytes of
  // each of the warp's 32 rows, 16-byte units swizzled: unit u of this lane's row, and of its places, as addresses.
  __device__ __forceinline__ uint32_t stage() const { return smem_u32(smem) + warp * 4096; }
  __device__ __forceinline__ uint32_t own(uint32_t base, int u) const { return (base + lane * 128 + ((lane & 7) << 4)) ^ (u << 4); }
  __device__ __forceinline__ uint32_t placed(uint32_t base, int k) const {
    return base + lane / 8 * 128 + (((lane % 8) ^ (lane / 8) ^ (4 * (k & 1))) << 4) + k * 512;
  }
  // Elements from a tensor's first to each place's first (rows that are not there: the warp's first row's, so that nothing has to branch).
  struct Places {
    int64_t off[8];
    __device__ __forceinline__ void init(int64_t mine, bool live, int lane) {
      const int64_t first = __shfl_sync(0xffffffffu, mine, 0);
      if (!live) mine = first;
#pragma unroll
      for (int k = 0; k < 8; ++k) off[k] = __shfl_sync(0xffffffffu, mine, 4 * k + lane / 8) + lane % 8 * 8;
    }
  };

  // The warp's queries to where the MMAs take them, times the sign of the scale; returns by what the scores of this lane's row are
  // scaled besides (8-bit caches: its power of two).
  __device__ __forceinline__ float put_queries(const Places& places, uint32_t mine) {
    constexpr int C = D / 64, AHEAD = C < 2 ? C : 2;    // 128-byte columns, and how many are asked for at once
    float up = 1.f, by = p.scale_log2 > 0.f ? 1.f : p.scale_log2 < 0.f ? -1.f : 0.f;
    const bool narrow = T::F8 && p.q_bf16;
    // where a column goes: to the stage and on to tensor memory, or to its place
    auto base = [&](int c) { return T::QT ? stage() : smem_u32(smem) + c * (kTreeRows * 128) + warp * 4096; };
    auto ask = [&](int c, int k) { return __ldg(reinterpret_cast<const uint4*>(p.q + places.off[k] + 64 * c)); };
    if (narrow) {
      float top = 0.f;
#pragma unroll 1
      for (int c = 0; c < C; ++c) {
        uint4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = ask(c, k);
#pragma unroll
        for (int k = 0; k < 8; ++k) st_shared(placed(base(0), k), x[k]);
        __syncwarp();
#pragma unroll 2
        for (int u = 0; u < 8; ++u) {
          const uint4 v = ld_shared(own(base(0), u));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = unpack2<true>(w[j]);
            top = max3(top, fabsf(f.x), fabsf(f.y));
          }
        }
        __syncwarp();
      }
      // 2^e <= top < 2^(e + 1); e is kept where both 2^e and 2^-e are normal (an infinite or NaN q stays one)
      const int e = min(max(static_cast<int>((__float_as_uint(top) >> 23) & 255u) - 127, -126), 126);
      up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
      by *= __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    }
    // this lane's row of a column, in place
    auto scale = [&](int c) {
      if (!narrow && p.scale_log2 > 0.f) return;
#pragma unroll 1
      for (int u = 0; u < 8; ++u) {
        const uint32_t at = own(base(c), u);
        const uint4 v = ld_shared(at);
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = T::BF16 || p.q_bf16 ? unpack2<true>(w[j]) : unpack2<false>(w[j]);
          w[j] = pack2<T::BF16>(f.x * by, f.y * by);
        }
        st_shared(at, make_uint4(w[0], w[1], w[2], w[3]));
      }
    };
#pragma unroll 1
    for (int c0 = 0; c0 < C; c0 += AHEAD) {
      uint4 x[AHEAD][8];
#pragma unroll
      for (int c = 0; c < AHEAD; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) x[c][k] = ask(c0 + c, k);
#pragma unroll
      for (int c = 0; c < AHEAD; ++c) {
#pragma unroll
        for (int k = 0; k < 8; ++k) st_shared(placed(base(c0 + c), k), x[c][k]);
        __syncwarp();
        scale(c0 + c);
        if constexpr (T::QT) {
          uint32_t w[32];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const uint4 v = ld_shared(own(base(0), u));
            w[4 * u] = v.x, w[4 * u + 1] = v.y, w[4 * u + 2] = v.z, w[4 * u + 3] = v.w;
          }
          tmem_st_32x32b_x32(mine + T::TMEM_Q + 32 * (c0 + c), w);
          __syncwarp();
        }
      }
    }
    if constexpr (T::QT) {
      tmem_wait_st();
      tc_fence_before();
    } else {
      fence_proxy_async_smem();
    }
    return up;
  }

  // S of 32 keys, what the row does not see as -inf.
  __device__ __forceinline__ void hide(uint32_t (&s)[32], uint32_t sees) {
    if (sees != ~0u) {
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (!(sees >> c & 1)) s[c] = 0xFF800000u;
    }
  }
  __device__ __forceinline__ float highest(const uint32_t (&s)[32]) {
    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int c = 0; c < 32; c += 2) top[c / 2 % 4] = max3(top[c / 2 % 4], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
    return max3(fmaxf(top[0], top[1]), top[2], top[3]);
  }
  // Of a tile; returns the maximum.
  __device__ __forceinline__ float scores(uint32_t (&s)[2][32], uint32_t at, uint64_t sees) {
    tmem_ld_32x32b_x32(at, s[0]);
    read_tmem(at + 32, s[1]);
    arrived(s[0]);
    hide(s[0], static_cast<uint32_t>(sees));
    hide(s[1], static_cast<uint32_t>(sees >> 32));
    return fmaxf(highest(s[0]), highest(s[1]));
  }

  // P of 32 keys in place of S, as (key, key + 1) pairs: for each 16 keys 8 columns of high parts, 8 of low ones. Adds to sum.
  __device__ __forceinline__ void weights(uint32_t (&s)[32], uint32_t at, float2 sc, float2 base, float2& sum) {
    uint32_t out[32];
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
      const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc, base);
      const float2 e = make_float2(exp2_approx(x.x), exp2_approx(x.y));
      sum = __fadd2_rn(sum, e);
      uint32_t hi;
      float2 back;
      if constexpr (T::BF16) {                          // towards zero: the upper halves
        hi = __byte_perm(__float_as_uint(e.x), __float_as_uint(e.y), 0x7632);
        back = make_float2(__uint_as_float(__float_as_uint(e.x) & 0xFFFF0000u), __uint_as_float(__float_as_uint(e.y) & 0xFFFF0000u));
      } else {
        hi = pack2<false>(e.x, e.y);
        back = unpack2<false>(hi);
      }
      out[c / 16 * 16 + c % 16 / 2] = hi;
      out[c / 16 * 16 + c % 16 / 2 + 8] = pack2<T::BF16>(e.x - back.x, e.y - back.y);
    }
    tmem_st_32x32b_x32(at, out);
  }

  // Infinite and NaN values that the row sees, in 32 of its channels from d on: those that were taken out of tiles that not all rows see
  // whole; and, as a weight that underflowed to 0 makes an infinity NaN, all of them where a channel is NaN.
  __device__ __noinline__ void add_odd(float* o, int d, const Walk<MODE, T::COST>& w, const Piece& x, uint64_t mask, bool all) const {
    for (int c = 0; c < 32; ++c)
      if (o[c] != o[c]) o[c] = 0.f;
    for (int i = x.begin; i < x.end; ++i) {
      const Tile t = tile(p, w.r, i);
      if (t.plain && !all) continue;
      uint64_t sees = visible(p, w.r, t, mask) & low_bits(t.end - t.k0);
      while (sees != 0) {
        const int key = t.k0 + __ffsll(static_cast<long long>(sees)) - 1;
        sees &= sees - 1;
        const int at = p.page.div(key), page = __ldg(p.pages + w.b * p.ldp + at);
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) continue;
        const uint8_t* row = p.v + page * p.page_stride + x.kvh * p.head_stride + static_cast<int64_t>(key - at * p.page.d) * p.token_stride;
        for (int c = 0; c < 32; ++c) {
          float v;
          if constexpr (T::F8) {
            v = (row[d + c] & 0x7F) == 0x7F ? NAN : 0.f;
          } else {
            const uint32_t bits = reinterpret_cast<const uint16_t*>(row)[d + c];
            v = unpack2<T::BF16>(bits).x;
          }
          if (!(fabsf(v) < INFINITY)) o[c] += v;
        }
      }
    }
  }

  // Pages up to the key `end` do not exist: an error where a node sees that far back. A window's tiles begin where a row without nodes would; all
  // nodes may see less, and their pages before that may be gone.
  __device__ __noinline__ void missing(const Request r, int end) const {
    int fewest = TL_TREE_NODES;
    for (int i = 0; i < r.n; ++i) fewest = min(fewest, __popcll(static_cast<uint64_t>(__ldg(p.masks + r.row0 + i)) & low_bits(r.n)));
    if (p.window == 0 || end > r.len - max(0, p.window - fewest)) set_status(p.status, TL_EDATA);
  }

  __device__ __forceinline__ void run() {
    Walk<MODE, T::COST> w;
    w.init(p, 2 * kKeys * T::ROW, MODE == kCluster ? warp == 0 : blockIdx.x == 0 && warp == 0);
    Piece x;
    uint32_t tiles = 0, pieces = 0;
    TreeCut cut{};
    const uint32_t mine = misc->tmem + (static_cast<uint32_t>(warp) << 21);      // this warp's 32 lanes
    // The piece's rows from 32 `first` on are this warp's: where two blocks share an SM, warps w and w + 2 of the second change places, so that
    // few rows of both keep all four schedulers at work.
    const int first = warp ^ ((misc->tmem & 0xFFFF) != 0 ? 2 : 0);
    while (ok && w.next(p, x)) {
      const int first_row = x.row_block * kTreeRows, rows = min(kTreeRows, w.r.n * p.group - first_row);
      const int mr = first * 32 + lane;
      const bool busy = first * 32 < rows, live = mr < rows;
      const int gr = first_row + (live ? mr : 0), node = static_cast<int>(p.group_div.div(gr)), head = x.kvh * p.group + gr - node * p.group;
      const int64_t token = static_cast<int64_t>(w.r.row0) + node;
      uint64_t mask = 0;
      float sc = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2), vs = 1.f;       // (its sign, or zero, is in the queries)
      if constexpr (T::F8) {
        sc *= __ldg(p.k_scale + x.kvh);
        vs = __ldg(p.v_scale + x.kvh);
      }
      if (live) mask = static_cast<uint64_t>(__ldg(p.masks + token)) & low_bits(w.r.n);
      if (busy) {
        Places places;
        places.init(token * p.ldq + static_cast<int64_t>(head) * D, live, lane);
        sc *= put_queries(places, mine);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&misc->q_full));
      float m = -INFINITY;
      float2 l = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int i = x.begin; i < x.end; ++i, ++tiles) {
        const uint32_t buf = tiles % T::SBUF;
        if (!wait(misc->s_full[buf], tiles / T::SBUF)) break;
        if (busy) {
          tc_fence_after();
          const uint32_t sb = mine + T::TMEM_S + buf * kKeys;
          const Tile t = tile(p, w.r, i);
          const uint64_t sees = t.plain ? ~0ull : visible(p, w.r, t, mask);
          uint32_t s[2][32];
          bool settled = false;
          for (;;) {
            const float top = scores(s, sb, sees) * sc;
            const bool grown = top > m + T::SLACK || (m == -INFINITY && top > m);
            if (i == x.begin) m = top;
            if (settled || i == x.begin || !__any_sync(0xffffffffu, grown)) break;
            // o and l are scaled down to the new maximum; the MMAs of the tile before add to o until they are done
            if (!wait(misc->pv_done[(tiles - 1) % T::SBUF], (tiles - 1) / T::SBUF)) break;
            tc_fence_after();
            const float f = grown ? faded(m - top) : 1.f;
            if (grown) m = top;
            l.x *= f, l.y *= f;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              read_tmem(mine + c, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st_32x32b_x32(mine + c, o);
            }
            settled = true;                             // the scores once more: they need not be kept meanwhile
          }
          if (!ok) break;
          const float base = T::POFF - (m == -INFINITY ? 0.f : m);
#pragma unroll
          for (int h = 0; h < 2; ++h) weights(s[h], sb + 32 * h, make_float2(sc, sc), make_float2(base, base), l);
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&misc->p_full[buf]));
      }
      if (!ok) break;
      if (!wait(misc->pv_done[(tiles - 1) % T::SBUF], (tiles - 1) / T::SBUF) || !wait(misc->loaded[pieces % kAhead], pieces / kAhead)) break;
      const bool odd = *const_cast<volatile int*>(&misc->flag[pieces % kAhead]) == static_cast<int>(pieces) + 1;
      if (warp == 0 && lane == 0) {
        volatile int* const bad = &misc->bad[pieces % kAhead];
        if (*bad != 0) missing(w.r, *bad), *bad = 0;
      }
      ++pieces;
      if (busy) {
        tc_fence_after();
        // a cluster's parts stay in the ring, which is at rest
        float* const part = MODE == kCluster ? reinterpret_cast<float*>(smem + T::OFF_SLOT)
                                             : p.partials + (static_cast<size_t>(2) * blockIdx.x + x.second) * tree_partial_floats(D);
        const float sum = l.x + l.y, inv = sum == 0.f ? 0.f : vs / sum;
        Places places;
        if (x.whole) places.init(token * p.ldo + static_cast<int64_t>(head) * D, live, lane);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          read_tmem(mine + c, o);
          float2 all[2] = {{0.f, 0.f}, {0.f, 0.f}};     // NaN where one of them is, or where infinities meet
#pragma unroll
          for (int e = 0; e < 32; e += 2) all[e / 2 % 2] = __fadd2_rn(all[e / 2 % 2], make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])));
          all[0] = __fadd2_rn(all[0], all[1]);
          const bool nan = !(all[0].x + all[0].y == all[0].x + all[0].y);
          if (live && (odd || nan) && sum == sum) {
            float f[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(o[e]);
            add_odd(f, c, w, x, mask, nan);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(f[e]);
          }
          if (!x.whole) {                               // [4 channels][row]: neighbouring rows side by side
            float4* const q = reinterpret_cast<float4*>(part + 2 * kTreeRows) + (c / 4) * kTreeRows + mr;
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              if (live)
                q[e / 4 * kTreeRows] = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]), __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
            continue;
          }
          const int half = c % 64 / 8;                  // 64 channels of 32 rows pass through shared memory
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f = __fmul2_rn(make_float2(__uint_as_float(o[e + 2 * k]), __uint_as_float(o[e + 2 * k + 1])), make_float2(inv, inv));
              v[k] = T::BF16 ? pack2<true>(f.x, f.y) : !T::F8 ? pack2<false>(f.x, f.y) : p.q_bf16 ? pack2<true>(f.x, f.y) : pack2<false>(f.x, f.y);
            }
            st_shared(own(stage(), half + e / 8), make_uint4(v[0], v[1], v[2], v[3]));
          }
          if (half == 0) continue;
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint4 v = ld_shared(placed(stage(), k));
            if (first * 32 + 4 * k + lane / 8 < rows) *reinterpret_cast<uint4*>(p.out + places.off[k] + c - 32) = v;
          }
          __syncwarp();
        }
        tc_fence_before();
        if (live) {
          if (x.whole) {
            if (p.lse != nullptr) p.lse[token * p.q_heads + head] = sum == 0.f ? -INFINITY : (m - T::POFF) * kLn2 + logf(sum);
          } else {
            part[mr] = m;
            part[kTreeRows + mr] = sum;
          }
        }
      }
      if (!x.whole && x.starts_here) cut = TreeCut{x.parts, w.r.row0, x.kvh, first_row, rows, vs};
    }
    if (MODE == kList && warp == 0 && lane == 0) p.cuts[blockIdx.x] = cut;
  }
};

// The blocks of a cluster join their parts, each some (row, four channels); all threads of all of them.
template <int CACHE, int D>
__device__ __forceinline__ void join_cluster(const TreeAttnParams& p, uint8_t* smem, const Walk<kCluster, Traits<CACHE, D>::COST>& w) {
  using T = Traits<CACHE, D>;
  const int size = 1 << p.cluster_log, rank = blockIdx.x & (size - 1);
  const int kvh = w.seg / p.row_blocks, first_row = (w.seg - kvh * p.row_blocks) * kTreeRows;
  const int rows = min(kTreeRows, w.r.n * p.group - first_row), padded = (rows + 31) & ~31;
  const uint32_t part = smem_u32(smem) + T::OFF_SLOT;
  float vs = 1.f;
  if constexpr (T::F8) vs = __ldg(p.v_scale + kvh);
  for (int i = rank * T::THREADS + static_cast<int>(threadIdx.x); i < padded * (D / 4); i += size * T::THREADS) {
    const int d4 = i / padded, r = i - d4 * padded;
    if (r >= rows) continue;
    float top = -INFINITY, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    // N blocks' parts with one latency
    auto take = [&](auto count, int from) {
      constexpr int N = decltype(count)::value;
      float m[N], s[N], most = top;
      float4 v[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        m[k] = attn::ld_cluster(part + 4 * r, from + k);
        s[k] = attn::ld_cluster(part + 4 * (kTreeRows + r), from + k);
        v[k] = attn::ld_cluster4(part + 4 * (2 * kTreeRows) + 16 * (d4 * kTreeRows + r), from + k);
        most = fmaxf(most, m[k]);
      }
      const float base = most == -INFINITY ? 0.f : most, f0 = faded(top - base);
      top = most;
      l *= f0, a.x *= f0, a.y *= f0, a.z *= f0, a.w *= f0;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (s[k] == 0.f) continue;                      // nothing was seen, or there was no tile: o is not what it should be
        const float f = faded(m[k] - base);
        l += f * s[k];
        a.x += f * v[k].x;
        a.y += f * v[k].y;
        a.z += f * v[k].z;
        a.w += f * v[k].w;
      }
    };
    if (size >= 8)
      for (int k = 0; k < size; k += 8) take(std::integral_constant<int, 8>{}, k);
    else if (size == 4)
      take(std::integral_constant<int, 4>{}, 0);
    else
      take(std::integral_constant<int, 2>{}, 0);
    const int gr = first_row + r, node = static_cast<int>(p.group_div.div(gr)), head = kvh * p.group + gr - node * p.group;
    const int64_t token = static_cast<int64_t>(w.r.row0) + node;
    const float inv = l == 0.f ? 0.f : vs / l;
    uint2 out;
    out.x = p.q_bf16 ? pack2<true>(a.x * inv, a.y * inv) : pack2<false>(a.x * inv, a.y * inv);
    out.y = p.q_bf16 ? pack2<true>(a.z * inv, a.w * inv) : pack2<false>(a.z * inv, a.w * inv);
    *reinterpret_cast<uint2*>(p.out + token * p.ldo + static_cast<int64_t>(head) * D + 4 * d4) = out;
    if (d4 == 0 && p.lse != nullptr) p.lse[token * p.q_heads + head] = l == 0.f ? -INFINITY : (top - T::POFF) * kLn2 + logf(l);
  }
}

template <int CACHE, int D, Mode MODE>
__global__ void __launch_bounds__(Traits<CACHE, D>::THREADS, Traits<CACHE, D>::BLOCKS) tree_attention_kernel(const __grid_constant__ TreeAttnParams p) {
  using T = Traits<CACHE, D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc<T>* const misc = reinterpret_cast<Misc<T>*>(smem + T::OFF_MISC);
  static_assert(sizeof(Misc<T>) <= 1024, "misc");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((smem_u32(smem) & 1023) != 0) {                  // the swizzle goes by addresses
    if (threadIdx.x == 0) set_status(p.status, TL_ECUDA);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < T::SLOTS; ++i) mbar_init(smem_u32(&misc->full[i]), 32), mbar_init(smem_u32(&misc->empty[i]), 1);
    for (int i = 0; i < T::SBUF; ++i) {
      mbar_init(smem_u32(&misc->s_full[i]), 1);
      mbar_init(smem_u32(&misc->p_full[i]), kSoftmaxWarps);
      mbar_init(smem_u32(&misc->pv_done[i]), 1);
    }
    mbar_init(smem_u32(&misc->q_full), kSoftmaxWarps);
    for (int i = 0; i < kAhead; ++i) mbar_init(smem_u32(&misc->loaded[i]), T::LOADERS), misc->flag[i] = misc->bad[i] = 0;
    misc->abort = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&misc->tmem), T::TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait_prior();
  if (warp < kSoftmaxWarps) {
    Softmax<CACHE, D, MODE> s{p, smem, misc, warp, lane};
    s.run();
  } else if (warp == kMmaWarp) {
    Mma<CACHE, D, MODE> m{p, smem, misc};
    m.run();
  } else {
    Loader<CACHE, D, MODE> l{p, smem, misc, warp - kLoadWarp, lane};
    l.run();
  }
  pdl_launch_dependents();
  if (MODE == kCluster && p.cluster_log > 0) {
    Walk<kCluster, T::COST> w;
    w.init(p, 0, false);
    if (w.more && warp < kSoftmaxWarps && (w.r.tiles >> p.cluster_log) == 0) {
      // a block without tiles says so
      Piece x;
      if (!w.next(p, x)) {
        float* const part = reinterpret_cast<float*>(smem + T::OFF_SLOT);
        part[threadIdx.x] = -INFINITY;
        part[kTreeRows + threadIdx.x] = 0.f;
      }
      w.more = true;
    }
    __syncwarp();
    cluster_sync();                                     // (all blocks meet, whatever each has read of the request)
    if (w.more) join_cluster<CACHE, D>(p, smem, w);
    cluster_sync();                                     // no block leaves while another reads its part
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(misc->tmem, T::TMEM);
  }
}

// ---- the second kernel: segments that were cut. Block x joins the one that begins in the share of block x of the first kernel,
// 32 channels of it; a thread takes them of a row, and where the rows need fewer warps than there are, those share the partials out.
constexpr int kJoinWarps = 8;

template <int D, bool F16>
__global__ void __launch_bounds__(kJoinWarps * 32) tree_join_kernel(const __grid_constant__ TreeAttnParams p) {
  constexpr float POFF = F16 ? Traits<kCacheF16, D>::POFF : Traits<kCacheBf16, D>::POFF;
  __shared__ float s_o[kJoinWarps][33][32];
  __shared__ float s_m[kJoinWarps][32];
  pdl_wait_prior();
  pdl_launch_dependents();
  const TreeCut c = p.cuts[blockIdx.x];
  if (c.parts == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row_warps = c.rows <= 32 ? 1 : c.rows <= 64 ? 2 : 4, share = kJoinWarps / row_warps;     // warps to 32 rows
  const int r = warp % row_warps * 32 + lane, turn = warp / row_warps, d4 = blockIdx.y * 8;
  auto part = [&](int i) { return p.partials + (static_cast<size_t>(2) * (blockIdx.x + i) + (i == 0)) * tree_partial_floats(D); };
  float top = -INFINITY, l = 0.f, a[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) a[e] = 0.f;
  if (r < c.rows) {
#pragma unroll 8
    for (int i = turn; i < c.parts; i += share) top = fmaxf(top, __ldcg(part(i) + r));
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll 2
    for (int i = turn; i < c.parts; i += share) {
      const float* const q = part(i);
      const float f = faded(__ldcg(q + r) - base);
      l += f * __ldcg(q + kTreeRows + r);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(q + 2 * kTreeRows) + (d4 + e) * kTreeRows + r);
        a[4 * e] += f * v.x;
        a[4 * e + 1] += f * v.y;
        a[4 * e + 2] += f * v.z;
        a[4 * e + 3] += f * v.w;
      }
    }
  }
  // the warps of the same rows: halves add to halves, in a fixed order
  for (int n = share / 2; n > 0; n /= 2) {
    if (turn >= n && turn < 2 * n) {
      s_m[warp][lane] = top;
      s_o[warp][32][lane] = l;
#pragma unroll
      for (int e = 0; e < 32; ++e) s_o[warp][e][lane] = a[e];
    }
    __syncthreads();
    if (turn < n) {
      const int other = warp + n * row_warps;
      const float m2 = s_m[other][lane], most = fmaxf(top, m2), base = most == -INFINITY ? 0.f : most;
      const float f1 = faded(top - base), f2 = faded(m2 - base);
      top = most;
      l = l * f1 + s_o[other][32][lane] * f2;
#pragma unroll
      for (int e = 0; e < 32; ++e) a[e] = a[e] * f1 + s_o[other][e][lane] * f2;
    }
    __syncthreads();
  }
  if (turn != 0 || r >= c.rows) return;
  const int gr = c.first_row + r, node = static_cast<int>(p.group_div.div(gr)), head = c.kvh * p.group + gr - node * p.group;
  const int64_t token = static_cast<int64_t>(c.row0) + node;
  const float inv = l == 0.f ? 0.f : c.v_scale / l;
  uint16_t* const to = p.out + token * p.ldo + static_cast<int64_t>(head) * D + 4 * d4;
#pragma unroll
  for (int e = 0; e < 32; e += 8) {
    uint32_t v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = p.q_bf16 ? pack2<true>(a[e + 2 * k] * inv, a[e + 2 * k + 1] * inv) : pack2<false>(a[e + 2 * k] * inv, a[e + 2 * k + 1] * inv);
    *reinterpret_cast<uint4*>(to + e) = make_uint4(v[0], v[1], v[2], v[3]);
  }
  if (blockIdx.y == 0 && p.lse != nullptr) p.lse[token * p.q_heads + head] = l == 0.f ? -INFINITY : (top - POFF) * kLn2 + logf(l);
}

template <int CACHE, int D>
cudaError_t launch(TreeAttnParams& p, int sms, cudaStream_t st) {
  using T = Traits<CACHE, D>;
  static int ready[64], at_once[64][kMaxClusterLog + 1];         // by device: how many clusters of 2^i blocks run at once
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto* const clusters = tree_attention_kernel<CACHE, D, kCluster>;
  if (__atomic_load_n(&ready[dev], __ATOMIC_ACQUIRE) == 0) {
    for (auto* kernel : {tree_attention_kernel<CACHE, D, kList>, clusters}) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM);
      if (e != cudaSuccess) return e;
    }
    e = cudaFuncSetAttribute(clusters, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    __atomic_store_n(&at_once[dev][0], sms * T::BLOCKS, __ATOMIC_RELAXED);
    for (int log = 1; log <= kMaxClusterLog; ++log) {
      cudaLaunchAttribute size;
      size.id = cudaLaunchAttributeClusterDimension;
      size.val.clusterDim.x = 1 << log, size.val.clusterDim.y = size.val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(1 << log), cfg.blockDim = dim3(T::THREADS), cfg.dynamicSmemBytes = T::SMEM;
      cfg.attrs = &size, cfg.numAttrs = 1;
      int n = 0;
      e = cudaOccupancyMaxActiveClusters(&n, clusters, &cfg);
      if (e != cudaSuccess) return e;
      __atomic_store_n(&at_once[dev][log], n, __ATOMIC_RELAXED);
    }
    __atomic_store_n(&ready[dev], 1, __ATOMIC_RELEASE);
  }
  const long long nodes = p.T < TL_TREE_NODES ? p.T : TL_TREE_NODES;
  const long long seen = p.window > 0 ? p.window + 15ll + p.sinks : p.capacity, keys = (seen < p.capacity ? seen : p.capacity) + nodes;
  const long long tiles = (keys + kKeys - 1) / kKeys + (p.sinks > 0);
  p.row_blocks = static_cast<int>((nodes * p.group + kTreeRows - 1) / kTreeRows);
  const long long segments = static_cast<long long>(p.B) * p.kv_heads * p.row_blocks;
  // Few segments of few tiles: a cluster each, of the most blocks that all run at once, while a block has more than one tile and
  // no more than some, where the list's equal shares and its more blocks win; of the up to seven segments that have sixteen blocks the
  // list makes so many parts that this is later. Lengths lie on the GPU, so keys are counted by the table's width, and nodes by T: a short request
  // behind a wide table gets what suits a long one (577 tokens, tables of 640, 4096 and from 32768 on: 12.1, 12.7, 16.5; 4000: 17.1, 17.1, 24.6;
  // 64 channels 8.9, 9.0, 14.0 and 11.5, 11.6, 28.4). One request of 577 tokens, 8 nodes: clusters 11.7 us (16 blocks for its 10 tiles: 14.5), the
  // list 15.1; 4000: 15.6 and 23.1, 64 channels 11.0 and 29.2; 16000: 28.2 and 32.1, 20.1 and 31.4; seven heads of 128 channels, 29000:
  // 34 and 40, four in 8 bits 38 and 32. Eight requests of 1000: two blocks each 22.4, the list 20.4.
  for (int log = kMaxClusterLog; log >= 0; --log) {
    const int c = 1 << log;
    if (segments > __atomic_load_n(&at_once[dev][log], __ATOMIC_RELAXED) || (log > 0 && tiles <= c)) continue;
    if (tiles > (log < kMaxClusterLog ? 10 : T::F8 ? 20 : 30) * c) break;
    p.cluster_log = log;
    return launch_pdl_cluster(clusters, dim3(static_cast<unsigned>(segments * c)), dim3(T::THREADS), T::SMEM, st, c, p);
  }
  long long grid = static_cast<long long>(sms) * T::BLOCKS;
  if (grid > kTreeMaxGrid) grid = kTreeMaxGrid;
  const long long most = segments * (tiles + T::COST);    // places that the list can have
  if (grid > most) grid = most;
  p.grid = static_cast<int>(grid);
  e = launch_pdl(tree_attention_kernel<CACHE, D, kList>, dim3(static_cast<unsigned>(grid)), dim3(T::THREADS), T::SMEM, st, p);
  if (e != cudaSuccess || grid == 1) return e;
  return launch_pdl(tree_join_kernel<D, !T::BF16>, dim3(static_cast<unsigned>(grid), D / 32), dim3(kJoinWarps * 32), 0, st, p);
}

template <int CACHE>
cudaError_t launch_dim(TreeAttnParams& p, int dim, int sms, cudaStream_t st) {
  switch (dim) {
    case 64: return launch<CACHE, 64>(p, sms, st);
    case 128: return launch<CACHE, 128>(p, sms, st);
    case 256: return launch<CACHE, 256>(p, sms, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tree
}  // namespace tl
