// The tiled product under the fused operators (gated block, cross entropy).
//
//   acc[m][n] = sum over k of A(m, k) * B(n, k)
//
// with the single schedule of nt_swap_kernel (two ring slots of 64-deep K
// tiles, v_mfma_f32_16x16x32), two additions, and an epilogue of its own:
//
//  * each operand lies in memory either with K contiguous (KC: element (r, k)
//    at p[r * pitch + k], as in the NT calls) or as K rows (KR: at
//    p[k * pitch + r]).  The gradients need the second: dx = dY W contracts
//    over W's rows, dW = dY^T x over the tokens.  Transposing them first
//    would read and write each operand once more;
//  * the B rows of a tile may come from two matrices in blocks of 16 (DUAL):
//    an even block holds gate rows and the odd block after it the same up
//    rows, so that one lane holds the gate and the up value of an element.
//
// A KR tile is kept in its slot as it lies in memory: 64 rows (k) of R
// values.  Its MFMA fragments are read with ds_read_b64_tr_b16, which gives
// lane l of each group of 16 lanes the l-th column of the 4 x 16 block whose
// rows' 8-byte pieces the group's lanes address; two of them make the eight
// consecutive k that a lane of the 16x16x32 MFMA holds.
//
// Pitches are multiples of 8 elements and operands start on 16 bytes (the
// host pads what does not), so every 16-byte granule is whole.
#pragma once

#include <type_traits>

#include "instances.hpp"

namespace pgemm {

enum class Lay { KC, KR };

typedef short s16x4 __attribute__((ext_vector_type(4)));
// a 16-byte piece at any even address: the hardware takes unaligned global accesses
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

struct FusedOperand {
  const uint16_t *p;
  const uint16_t *p2;  // DUAL: the second matrix (same pitch)
  int pitch;           // elements; a multiple of 8
  int rows;            // output rows (columns of a KR operand) inside the matrix
};

struct FusedProduct {
  FusedOperand a, b;
  int M, N, K;  // N counts output columns (of one matrix when DUAL)
  int tiles_m, tiles_n, group_m;
  int m_base, n_base;  // of the first tile
  int k_chunk;  // K of a piece (a multiple of 64), or K
  int piece;    // set in the kernel: which piece this workgroup does
};

// Granules of a KR tile: 16 bytes of a k row; the row's 32-byte pairs are
// permuted by XOR with f(k), so that the sixteen k rows that a transposing
// read touches fall on different banks.
template <int R>
struct KRows {
  static constexpr int CPR = R / 8;          // granules per k row
  static constexpr int ROW_BYTES = R * 2;
  static constexpr int RPI = kWave / CPR;    // k rows per load instruction
  static constexpr int FMASK = R >= 256 ? 3 : 1;
  __device__ __forceinline__ static int f(int k) { return (k & 3) | (((k >> 3) & FMASK) << 2); }
};

// Direct-to-LDS loads that the compiler does not see as such.
//
// It takes every LDS read that follows a direct-to-LDS load for a possible
// reader of what that load brings.  Plain reads it can tell apart by their
// type; the transposing reads have none, and each would wait for all loads in
// flight (s_waitcnt vmcnt(0)), those of the next but one K tile included: that
// took 2.0 us a K tile of 256 x 256 x 64 instead of 1.6.  So the loads of
// kernels with transposing reads are inline assembly, which returns nothing in
// registers, and their waits are explicit: UntrackedWait counts them.  M0, the
// LDS address, is set by the first of four and read by the other three;
// nothing between them writes it (tests/test_fused_asm.py).
typedef int rsrc_words __attribute__((ext_vector_type(4)));

__device__ __forceinline__ rsrc_words make_rsrc_words(const char *base, uint32_t bytes) {
  const uint64_t v = reinterpret_cast<uint64_t>(base);
  return rsrc_words{(int)(uint32_t)v, (int)(uint32_t)(v >> 32) & 0xffff, (int)bytes, kRsrcWord3};
}

template <int G>
__device__ __forceinline__ void load_lds_x4_untracked(rsrc_words rsrc, const char *lds_base, uint32_t voffset) {
  if constexpr (G == 0) {
    const uint32_t lds = (uint32_t)(uintptr_t)(lds_void *)lds_base;
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :
                 : "v"(voffset), "s"(rsrc), "s"(lds)
                 : "memory");
  } else {
    asm volatile("buffer_load_dwordx4 %0, %1, 0 offen offset:%c2 lds"
                 :
                 : "v"(voffset - 1024u * G), "s"(rsrc), "n"(1024 * G)
                 : "memory");
  }
}

// s_waitcnt vmcnt(N) that the compiler keeps though it knows of no load.
template <int N>
__device__ __forceinline__ void wait_vmcnt_untracked() {
  asm volatile("s_waitcnt vmcnt(%c0)" : : "n"(N) : "memory");
}

__device__ __forceinline__ const char *wave_uniform(const char *p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
  return reinterpret_cast<const char *>((uint64_t)hi << 32 | lo);
}

// Fills ring slots with direct-to-LDS loads.  The first half of the waves
// load the A tile, the second half the B tile, PER instructions each; what a
// lane adds to the tile's start is worked out once per instruction.  The
// buffer resource is remade for every K tile: its base moves along K, so K
// rows of any number and pitch stay inside 32-bit offsets.
template <class G, Lay LA, Lay LB, bool DUAL>
struct FusedLoader {
  static constexpr int PER = G::PER_LOADER;
  static constexpr int WAVES = G::CW;
  static constexpr int BK = G::BK;
  static constexpr int A_BYTES = G::BM * BK * 2;
  static constexpr int SLOT_BYTES = (G::BM + G::BN) * BK * 2;
  static_assert(BK == 64 && WAVES % 2 == 0 && PER * (WAVES / 2) * 1024 == A_BYTES && G::BM == G::BN,
                "half of the waves load each operand");
  static_assert(PER % 4 == 0, "instruction parity and the gate/up blocks follow i alone");

  const char *base, *base2;  // the tile's first element at k = 0
  uint32_t vo[PER];          // bytes from there per instruction, this lane
  int lk[2];                 // KC: the lane's first k within the tile, by instruction parity
  int64_t step;              // bytes from one K tile to the next
  uint32_t span;             // KC: bytes of the tile's rows; KR: bytes of a k row
  uint32_t cut;              // KR: bytes before the tile's first column
  int K;
  bool kc;

  static constexpr bool UNTRACKED = LA == Lay::KR || LB == Lay::KR;
  static_assert(!(UNTRACKED && DUAL), "two matrices have K contiguous");
  using Rsrc = std::conditional_t<UNTRACKED, rsrc_words, __amdgpu_buffer_rsrc_t>;
  struct Tile {
    Rsrc r, r2;
    int rem;  // K left from the tile's first k
  };

  __device__ __forceinline__ static Rsrc resource(const char *p, uint32_t bytes) {
    if constexpr (UNTRACKED)
      return make_rsrc_words(p, bytes);
    else
      return make_rsrc(p, bytes);
  }
  template <int N>
  __device__ __forceinline__ static void wait() {
    if constexpr (UNTRACKED)
      wait_vmcnt_untracked<N>();
    else
      wait_vmcnt<N>();
  }
  template <int I>
  __device__ __forceinline__ static void load(const Rsrc &r, char *dst, uint32_t v) {
    if constexpr (UNTRACKED)
      load_lds_x4_untracked<I>(r, dst, v);
    else
      load_lds_x4<I>(r, dst, v, 0);
  }

  template <Lay L, int R, bool TWO>
  __device__ __forceinline__ void lay_out(const FusedOperand &o, int r0, int first) {
    const int lane = threadIdx.x & (kWave - 1);
    const uint32_t pb = (uint32_t)o.pitch * 2u;
    kc = L == Lay::KC;
    if constexpr (L == Lay::KC) {
      constexpr int RR = TWO ? R / 2 : R;  // rows of one matrix; those past its edge read zero
      const int have = o.rows - r0 < RR ? o.rows - r0 : RR;
      base = reinterpret_cast<const char *>(o.p + (int64_t)r0 * o.pitch);
      base2 = TWO ? reinterpret_cast<const char *>(o.p2 + (int64_t)r0 * o.pitch) : base;
      span = (uint32_t)have * pb;
      cut = 0;
      step = BK * 2;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int row = (first + i) * (kWave / 8) + lane / 8;
        const int chunk = (lane % 8) ^ RingRow<BK>::swz(row);
        // TWO: blocks of 16 tile rows alternate between the two matrices
        const int mr = TWO ? (row >> 5) * 16 + (row & 15) : row;
        vo[i] = (uint32_t)mr * pb + (uint32_t)chunk * 16u;
        if (i < 2) lk[i] = chunk * 8;
      }
    } else {
      using KR = KRows<R>;
      base = reinterpret_cast<const char *>(o.p + r0);
      base2 = base;
      span = pb;
      cut = (uint32_t)r0 * 2u;
      step = (int64_t)BK * pb;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int k = (first + i) * KR::RPI + lane / KR::CPR;
        const int chunk = (lane % KR::CPR) ^ (KR::f(k) << 1);
        vo[i] = (uint32_t)k * pb + (uint32_t)chunk * 16u;
      }
      lk[0] = lk[1] = -1;
    }
  }

  __device__ __forceinline__ void init(const FusedProduct &g, int m0, int n0, int wave, int k_end) {
    K = k_end;
    if (wave < WAVES / 2)
      lay_out<LA, G::BM, false>(g.a, m0, wave * PER);
    else
      lay_out<LB, G::BN, DUAL>(g.b, n0, (wave - WAVES / 2) * PER);
    // one operand per wave: the same in every lane, which the compiler cannot
    // see through the choice above (it would loop over the lanes at each load)
    base = wave_uniform(base);
    base2 = DUAL ? wave_uniform(base2) : base;
    step = (int64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)step);
    span = (uint32_t)__builtin_amdgcn_readfirstlane((int)span);
    cut = (uint32_t)__builtin_amdgcn_readfirstlane((int)cut);
    kc = __builtin_amdgcn_readfirstlane((int)kc) != 0;
    // five wait states between these and a load that reads them: the compiler
    // does not look into the untracked ones
    if constexpr (UNTRACKED) asm volatile("s_nop 4");
  }

  // The resource of K tile t (past the end: of no bytes, every lane reads zero).
  __device__ __forceinline__ Tile tile(int t) const {
    Tile s;
    const int64_t k0 = (int64_t)t * BK;
    const int64_t left = K - k0;
    s.rem = left > 0 ? (int)left : 0;
    const int64_t off = (int64_t)t * step;
    uint32_t bytes;
    if (kc)
      bytes = span - (uint32_t)(k0 * 2);
    else
      bytes = (uint32_t)(s.rem < BK ? s.rem : BK) * span - cut;
    if (s.rem == 0) bytes = 0;
    s.r = resource(base + off, bytes);
    s.r2 = DUAL ? resource(base2 + off, bytes) : s.r;
    return s;
  }

  // Instruction i of this wave's share of the tile, into `slot`.
  __device__ __forceinline__ void load_one(char *slot, int wave, const Tile &s, int i) const {
    uint32_t v = vo[i];
    if (lk[i & 1] >= s.rem) v = kOobOffset;
    char *dst = slot + (wave * PER + (i & ~3)) * (kWave * 16);
    const Rsrc r = DUAL && ((i >> 1) & 1) ? s.r2 : s.r;
    switch (i & 3) {
      case 0: load<0>(r, dst, v); break;
      case 1: load<1>(r, dst, v); break;
      case 2: load<2>(r, dst, v); break;
      default: load<3>(r, dst, v); break;
    }
  }
};

template <class Loader>
struct FusedRefill {
  const Loader &ld;
  char *slot;
  int wave;
  const typename Loader::Tile &s;
  int skip;  // instructions of the share issued before
  __device__ __forceinline__ void operator()(int i) const { ld.load_one(slot, wave, s, i + skip); }
};

// Where a lane reads its fragments of one operand: the blocks of 16 output
// rows of this wave, k32 step kk of the slot.
template <Lay L, int R>
struct FragSource {
  uint32_t off;  // KC: the lane's row; KR: the lane's k row and 8-byte piece
  int x;         // KC: chunk swizzle; KR: 32-byte pair permutation
  int chunk;
  int b0;        // the wave's first block
  __device__ __forceinline__ void init(int row0, int lane) {
    b0 = row0 / 16;
    if constexpr (L == Lay::KC) {
      const int r = lane & 15;
      off = (uint32_t)(row0 + r) * RingRow<64>::ROW_BYTES;
      x = RingRow<64>::swz(r);
      chunk = lane >> 4;
    } else {
      const int g = lane >> 4, q = lane & 15;
      off = (uint32_t)(8 * g + q / 4) * KRows<R>::ROW_BYTES + (q & 3) * 8;
      x = KRows<R>::f(8 * g + q / 4);
      chunk = 0;
    }
  }
  // block j, step kk, from the operand's part of the slot
  __device__ __forceinline__ u32x4 read(const char *part, int j, int kk) const {
    if constexpr (L == Lay::KC) {
      return *reinterpret_cast<const u32x4 *>(part + off + 16 * j * RingRow<64>::ROW_BYTES +
                                              (((4 * kk + chunk) ^ x) * 16));
    } else {
      constexpr int RB = KRows<R>::ROW_BYTES;
      const char *p = part + off + (uint32_t)(((b0 + j) ^ x) * 32) + kk * 32 * RB;
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p));
      const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * RB)));
      return u32x4{lo[0], lo[1], hi[0], hi[1]};
    }
  }
};

// The large tile (64 MFMAs per wave and step) runs nt_swap_kernel's split
// barriers with its placement; the small one (8) a single barrier at the
// start of a K tile's second step, after which the slot's refill is issued.
// Every K tile runs the same two steps, the last included: its refill reads
// zeros, and the fragments it reads ahead are not used.
//
// Large products are bound by the matrix units at the board's power limit:
// logits of 8192 x 65536 x 4096 in bf16 2980 us (1.48 PFLOP/s) with the softmax
// statistics and 2 x 1610 (1.37) with their derivative, dx and dW (one and two
// operands down the rows) 2 x 1545 and 2 x 1560 (1.42 and 1.41).  Small tiles are
// bound by what L2 gives, 32 KiB a CU and K tile, and all of them by the 6 to
// 12 us that filling the ring and storing a tile take when K is short: logits
// of 1021 x 50021 x 1000 in f16 150 us (0.68 PFLOP/s).
template <typename T, class G, Lay LA, Lay LB, bool DUAL, class Epi>
__global__ void __launch_bounds__(G::THREADS, G::OCC) fused_kernel(FusedProduct g, typename Epi::Args ea) {
  using Loader = FusedLoader<G, LA, LB, DUAL>;
  using W = WaveTile<T, G::WM, G::WN, G::BK>;
  constexpr int S = G::S, PER = Loader::PER, NR = W::TM + W::TN;
  static_assert(G::P == 0 && W::NK == 2, "slots of two k32 steps");
  extern __shared__ __attribute__((aligned(16))) char smem[];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int bm, bn, split;
  block_work(blockIdx.x, gridDim.x, g.tiles_m, g.tiles_n, g.group_m, &bm, &bn, &split);
  constexpr int ON = DUAL ? G::BN / 2 : G::BN;  // output columns of a tile
  const int m0 = g.m_base + bm * G::BM, n0 = g.n_base + bn * ON;
  const int wm = wave / G::WGN, wn = wave % G::WGN;
  g.piece = split;
  const int64_t k_end = ((int64_t)split + 1) * g.k_chunk;
  const int k_last = k_end < g.K ? (int)k_end : g.K;
  const int t0 = split * (g.k_chunk / G::BK);  // first K tile
  const int n_k = (int)(((int64_t)k_last + G::BK - 1) / G::BK) - t0;

  Loader ld;
  ld.init(g, m0, n0, wave, k_last);
  FragSource<LA, G::BM> fa;
  FragSource<LB, G::BN> fb;
  fa.init(wm * G::WM, lane);
  fb.init(wn * G::WN, lane);
  auto slot_ptr = [&](int s) { return smem + s * Loader::SLOT_BYTES; };
  typename W::Frags f[2];
  auto read = [&](typename W::Frags &to, int s, int kk, int r) __attribute__((always_inline)) {
    if (r < W::TN)
      to.b[r] = fb.read(slot_ptr(s) + Loader::A_BYTES, r, kk);
    else
      to.a[r - W::TN] = fa.read(slot_ptr(s), r - W::TN, kk);
  };

  W w;
  w.zero();
  for (int j = 0; j < S; ++j) {
    const typename Loader::Tile s = ld.tile(t0 + j);
#pragma unroll
    for (int i = 0; i < PER; ++i) ld.load_one(slot_ptr(j), wave, s, i);
  }
  Loader::template wait<(S - 1) * PER>();
  lds_barrier();
  if (n_k > 0) {
#pragma unroll
    for (int r = 0; r < NR; ++r) read(f[0], 0, 0, r);
  }
  for (int t = 0; t < n_k; ++t) {
    const int s = t % S;
    const typename Loader::Tile nt = ld.tile(t0 + t + S);
    auto rd1 = [&](int r) __attribute__((always_inline)) { read(f[1], s, 1, r); };
    auto rd0 = [&](int r) __attribute__((always_inline)) { read(f[0], (t + 1) % S, 0, r); };
    if constexpr (W::TM * W::TN == 64) {
      static_assert(S == 2, "the placement refills the slot of this tile");
      using Pl = SplitSyncPlacement<64>;
      static_assert(PER == Pl::NLA + Pl::NLB, "every load of the wave's share is placed");
      auto war = []() __attribute__((always_inline)) { lds_barrier(); };
      auto raw = []() __attribute__((always_inline)) {
        Loader::template wait<PER>();
        __builtin_amdgcn_s_barrier();
      };
      w.template sched_step<Pl::RA0, Pl::REA, NR, Pl::LA0, Pl::LEA, Pl::NLA, Pl::WAR>(
          f[0], rd1, FusedRefill<Loader>{ld, slot_ptr(s), wave, nt, 0}, war);
      w.template sched_step<Pl::RB0, Pl::REB, NR, Pl::LB0, Pl::LEB, Pl::NLB, Pl::RAW>(
          f[1], rd0, FusedRefill<Loader>{ld, slot_ptr(s), wave, nt, Pl::NLA}, raw);
    } else {
      constexpr int NM = W::TM * W::TN;
      static_assert(NR <= NM && NM % PER == 0, "reads and loads fit in a step");
      NoLoads none;
      auto no_sync = []() __attribute__((always_inline)) {};
      w.template sched_step<0, 1, NR, 0, 1, 0, -1>(f[0], rd1, none, no_sync);
      Loader::template wait<(S - 2) * PER>();  // tile t + 1 landed
      lds_barrier();    // and slot s is free
      w.template sched_step<0, 1, NR, NM / PER - 1, NM / PER, PER, -1>(
          f[1], rd0, FusedRefill<Loader>{ld, slot_ptr(s), wave, nt, 0}, no_sync);
    }
  }
  Loader::template wait<0>();  // loads past the end (zeros) land before the ring is reused
  w.settle();
  __syncthreads();
  typename Epi::template Run<T, G, W>{}(w, ea, g, smem, m0, n0, wm, wn, lane, tid);
}

}  // namespace pgemm
