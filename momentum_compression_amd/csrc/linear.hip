// Matrix products of 16-bit elements with an epilogue, on the matrix cores.
//
// out[r][c] = sum over k of R(r, k) C(c, k).  The columns' operand C is the
// matrix instruction's A, so that a lane's registers hold eight consecutive
// columns of one row of the result (16 bytes of it) when A's rows are read in
// perm_row() order.  Each operand comes with k contiguous (read as rows of the
// tile in LDS) or with its own index contiguous (read by transposing LDS reads),
// so the product of a layer and both of its gradients need no transposed copies.
#include <type_traits>

#include "activation.h"
#include "attention.h"

namespace onebit {
namespace {

using u32x4 = uint32_t __attribute__((ext_vector_type(4)));

// Orders a wave's own writes to LDS before its reads of what other lanes wrote.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

constexpr int kDeep = 64;  // of the summed index a tile: rows of a whole cache line
constexpr int64_t kCUs = 256;

// Eight values of a row of the result, `n` of them inside, at any element address.
// Whole 32-bit words are moved: what single elements are merged with is moved by
// elements.
template <typename S>
struct Words8 {
    typedef uint32_t Any __attribute__((ext_vector_type(2 * sizeof(S)), aligned(sizeof(S))));
};

template <typename S>
__device__ __forceinline__ void load_row8(float out[8], const S* p, int64_t n) {
    if (n >= 8) {
        const auto w = *reinterpret_cast<const typename Words8<S>::Any*>(p);
        S x[8];
        __builtin_memcpy(x, &w, sizeof(x));
#pragma unroll
        for (int e = 0; e < 8; ++e) out[e] = (float)x[e];
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = e < 7 && e < n ? (float)p[e] : 0.0f;
}

template <typename S>
__device__ __forceinline__ void store_row8(S* p, const float v[8], int64_t n) {
    if (n >= 8) {
        S x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (S)v[e];
        typename Words8<S>::Any w;
        __builtin_memcpy(&w, x, sizeof(x));
        *reinterpret_cast<typename Words8<S>::Any*>(p) = w;
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n) p[e] = (S)v[e];
}

// The bias of columns c ... c + 7.
template <typename T>
__device__ __forceinline__ void load_bias(float b[8], const ProductOut& o, int64_t c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = 0.0f;
    if (!o.bias || c >= o.cols) return;
    if (o.bias_wide) load_row8(b, (const float*)o.bias + c, o.cols - c);
    else load_row8(b, (const T*)o.bias + c, o.cols - c);
}

// The epilogue for columns c ... c + 7 of row r.
template <int ACT, typename S>
__device__ __forceinline__ void emit8(const ProductOut& o, int64_t r, int64_t c, const float b[8],
                                      float z[8]) {
    const int64_t n = o.cols - c;
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] += b[e];
    if (o.pre) store_row8((S*)o.pre + r * o.ld_pre + c, z, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = activate<ACT>(z[e]);
    if (o.residual) {
        float v[8];
        load_row8(v, (const S*)o.residual + r * o.ld_r + c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] += v[e];
    }
    S* to = (S*)o.out + r * o.ld + c;
    if (o.accumulate) {
        float v[8];
        load_row8(v, (const S*)to, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] += v[e];
    }
    store_row8(to, z, n);
}

// f with the activation as a constant.
template <typename F>
__host__ __device__ __forceinline__ void with_act(int32_t act, F&& f) {
    switch (act) {
        case ONEBIT_RELU: return f(std::integral_constant<int, ONEBIT_RELU>{});
        case ONEBIT_GELU: return f(std::integral_constant<int, ONEBIT_GELU>{});
        case ONEBIT_GELU_TANH: return f(std::integral_constant<int, ONEBIT_GELU_TANH>{});
        case ONEBIT_SILU: return f(std::integral_constant<int, ONEBIT_SILU>{});
        default: return f(std::integral_constant<int, ONEBIT_NONE>{});
    }
}

// One operand's tiles: TILE of its index by kDeep of the summed one.  By rows: TILE
// rows of kDeep elements in LDS; otherwise kDeep rows of TILE elements.  The 16-byte
// chunks of a row are xored with bits of the row's number, so that a read of 16
// rows' chunks, or a transposing read of 4 rows by 4 chunks, meets every bank once.
// A tile comes in pieces of 16 bytes a lane, which lie side by side in LDS: the
// lane asks for the chunk that the xor puts there.  What lies past the matrix reads
// as 0: such chunks get an offset past the buffer's end.
template <typename T, bool ROWS, int TILE, int WAVES>
struct Operand {
    static constexpr int kChunks = ROWS ? kDeep / 8 : TILE / 8;  // of a row in LDS
    static constexpr int kRowsAtOnce = 64 / kChunks * WAVES;
    static constexpr int kPer = TILE * kDeep * 2 / (1024 * WAVES);
    static constexpr int kBytes = TILE * kDeep * 2;
    static constexpr int kPeriod = ROWS ? 16 : 4;  // of the xor, in rows
    static_assert(kPer >= 1 && 64 % kChunks == 0 && kRowsAtOnce % kPeriod == 0, "whole pieces");
    static_assert(ROWS ? kChunks == 8 : kChunks >= 16, "the xor's layouts");
    const char* base;
    uint32_t stride, at;  // in bytes
    int64_t rest;         // from the first part to the second
    int32_t count;        // of the operand's index from the tile's first on
    int32_t mine;         // by rows: the lane's first k in a tile
    int32_t row0;         // the lane's first row in LDS
    int32_t past;         // else: of its eight columns, those past the row's end
    int64_t length;       // of a contiguous row: elements that may be read

    static __device__ __forceinline__ int swizzled(int row, int chunk) {
        if (!ROWS) return chunk ^ ((row & 3) << 2);
        return chunk ^ swizzle<64>(row);
    }
    __device__ __forceinline__ Operand(const ProductIn& in, int64_t first, int64_t extent, int wave,
                                       int lane) {
        const int row = wave * (64 / kChunks) + lane / kChunks;
        const int chunk = swizzled(row, lane % kChunks);  // the same kRowsAtOnce rows on
        stride = (uint32_t)in.ld * 2;
        const int64_t left = extent - first;
        count = left < TILE ? (int32_t)left : TILE;
        rest = in.rest;
        base = (const char*)in.p + (ROWS ? first * in.ld * 2 : first * 2);
        at = (uint32_t)row * stride + 16 * chunk;
        mine = 8 * chunk;
        row0 = row;
        length = in.row;
        past = past_end(first + mine, length);
        if (!ROWS && 8 * chunk >= count) at = 0x80000000u;
    }
    // Where the tile from k0 on begins, in the first part or the second.
    __device__ __forceinline__ const char* start(int64_t k0, bool second) const {
        return base + (ROWS ? k0 * 2 : k0 * stride) + (second ? rest : 0);
    }
    // The buffer of that tile and the lane's offset in it.
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(int64_t k0, bool second, int64_t depth,
                                                             uint32_t& off) const {
        const int64_t left = depth - k0;
        const char* from = start(k0, second);
        const int32_t deep = left < kDeep ? (int32_t)left : kDeep;
        // rows are made of whole chunks
        const uint32_t bytes =
            deep <= 0 ? 0u
            : ROWS    ? (uint32_t)(count - 1) * stride + (uint32_t)((deep + 7) & ~7) * 2
                      : (uint32_t)(deep - 1) * stride + (uint32_t)((count + 7) & ~7) * 2;
        off = ROWS && mine >= deep ? 0x80000000u : at;
        return __builtin_amdgcn_make_buffer_rsrc((void*)from, 0, (int)bytes, 0x00027000);
    }
    // Piece x of a tile, memory to LDS without registers between.
    __device__ __forceinline__ void load(char* tile, int x, __amdgpu_buffer_rsrc_t rsrc,
                                         uint32_t off, int wave) const {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc, (__attribute__((address_space(3))) void*)(tile + (x * WAVES + wave) * 1024), 16,
            (int)(off + (uint32_t)(x * kRowsAtOnce) * stride), 0, 0, 0);
    }
    // The same into registers.
    __device__ __forceinline__ u32x4 fetch(int x, __amdgpu_buffer_rsrc_t rsrc, uint32_t off) const {
        return __builtin_amdgcn_raw_buffer_load_b128(
            rsrc, (int)(off + (uint32_t)(x * kRowsAtOnce) * stride), 0, 0);
    }
    // Rows that lie anywhere and end anywhere (of eight elements or more): how many
    // of the lane's eight elements lie past the row's end, in the tile from k0 on.
    __device__ __forceinline__ int32_t over_of(int64_t k0) const {
        return ROWS ? past_end(k0 + mine, length) : past;
    }
    // Piece x of such a tile: where a row ends inside the lane's eight elements, the
    // row's last eight.
    __device__ __forceinline__ u32x4 fetch_any(int x, int64_t k0, bool second, int64_t depth,
                                               int32_t over) const {
        const int row = row0 + x * kRowsAtOnce;
        u32x4 v = {};
        if (over < 8 && (ROWS ? row < count : k0 + row < depth)) {
            typedef u32x4 Any __attribute__((aligned(2)));
            const char* from = start(k0, second) + (int64_t)row * stride + 2 * (mine - over);
            v = *reinterpret_cast<const Any*>(from);
        }
        return v;
    }
    // What fetch_any brought, moved down by `over` elements, zeros behind them.  Not
    // before it is needed: it waits for the load.
    static __device__ __forceinline__ u32x4 moved(u32x4 v, int32_t over) {
        if (!__any(over > 0 && over < 8)) return v;
        uint64_t lo = v[0] | (uint64_t)v[1] << 32, hi = v[2] | (uint64_t)v[3] << 32;
        if (over >= 4) {
            lo = hi;
            hi = 0;
        }
        const int bits = 16 * (over & 3);
        if (bits) {
            lo = lo >> bits | hi << (64 - bits);
            hi >>= bits;
        }
        return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
    }
    static __device__ __forceinline__ void put(char* tile, int x, u32x4 held, int wave, int lane) {
        *reinterpret_cast<u32x4*>(tile + (x * WAVES + wave) * 1024 + lane * 16) = held;
    }
    // 32 of the operand's index from `first` on, k from 16 kc on; PERM: the
    // order of perm_row().
    template <bool PERM>
    static __device__ __forceinline__ typename Mma<T>::x8 frag(const char* tile, int first, int kc,
                                                               int lane) {
        if (ROWS) {
            const int row = first + (PERM ? perm_row(lane & 31) : lane & 31);
            return *reinterpret_cast<const typename Mma<T>::x8*>(
                tile + row * (kDeep * 2) + (swizzled(row, 2 * kc + (lane >> 5)) << 4));
        }
        // of 16 lanes, lane i reads four elements of k row i / 4; swapping the
        // middle two groups of four permutes what the lanes get
        const int i = lane & 15;
        const int group = PERM ? ((i & 1) << 1) | ((i >> 1) & 1) : i & 3;
        const int row = 16 * kc + 8 * (lane >> 5) + (i >> 2);
        const int chunk = first / 8 + 2 * ((lane >> 4) & 1) + (group >> 1);
        const auto lo = read_tr<T>(tile + row * (TILE * 2) + (swizzled(row, chunk) << 4) +
                                   8 * (group & 1));
        const auto hi = read_tr<T>(tile + (row + 4) * (TILE * 2) + (swizzled(row + 4, chunk) << 4) +
                                   8 * (group & 1));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

struct ProductArgs {
    ProductIn a, b;       // columns' and rows' operand
    ProductOut out;
    float* parts;         // [splits][rows][padded] of a divided sum, or nullptr
    int64_t depth, padded;
    int32_t steps, half;  // of kDeep in the whole sum and in its first parts
    int32_t tiles_a, tiles_b, splits;
};

// A workgroup's tile.  Workgroups go to the 8 XCDs in turn: those of one XCD get
// consecutive tiles, and consecutive tiles are blocks of kBand columns' tiles, so
// that an XCD's L2 serves both operands several times.
constexpr uint32_t kBand = 8;
__device__ __forceinline__ void tile_of(const ProductArgs& p, uint32_t& ta, uint32_t& tb,
                                        uint32_t& split) {
    const uint32_t tiles = (uint32_t)p.tiles_a * p.tiles_b;
    split = blockIdx.x / tiles;
    uint32_t id = blockIdx.x % tiles;
    const uint32_t even = tiles / 8;
    if (id < even * 8) id = (id & 7) * even + (id >> 3);
    const uint32_t band = id / (kBand * p.tiles_b), left = p.tiles_a - band * kBand;
    const uint32_t wide = left < kBand ? left : kBand, in = id - band * kBand * p.tiles_b;
    ta = band * kBand + in % wide;
    tb = in / wide;
}

// A barrier that shows all waves the tiles whose loads they issued before, but for
// the last LOADS of each: a wave waits for its own first.
template <int LOADS>
__device__ __forceinline__ void step_barrier() {
    // its reads of LDS too: other waves replace what they read
    __builtin_amdgcn_s_waitcnt(0x0070 | (LOADS & 15) | ((LOADS >> 4) << 14));
    __syncthreads();
}

// Rows of a wave's part of the result on their way through LDS: the floats between
// two of them, so that 16 rows' pieces of 16 bytes meet every bank once.
template <int COLS>
constexpr int out_pitch() {
    return COLS + 4;
}

constexpr int kAhead = 3;  // tiles in LDS of a product that does not fill the GPU
template <int TA, int TB, int WA, int WB>
constexpr size_t product_lds(bool ahead) {
    const size_t tiles = (size_t)(TA + TB) * kDeep * 2 * (ahead ? kAhead : 2);
    const size_t rows = (size_t)WA * WB * 32 * out_pitch<TA / WA>() * sizeof(float);
    return tiles > rows ? tiles : rows;
}

// WA x WB waves of TA columns by TB rows of the result, two tiles of kDeep in LDS.
//
// A step multiplies a tile in parts of 16 k; the fragments of a part are read
// between the products of the part before it, the first of a tile after the step's
// one barrier, which stands before the last part of the tile before.  Behind that
// barrier the tile that was read is replaced, half of it among the products of that
// part and half among those of the next: a burst of loads would hold up the waves,
// as the loads of a CU pass at 64 bytes a cycle.  (8192^3 bf16: 814 to 850 us, 1290 to
// 1350 TFLOP/s, the matrix unit busy three quarters of the time; 8192 x 4096 over 1024:
// 69 to 73 us; with a GELU and `pre` 86 to 92, as nothing runs beside the epilogue of a CU's
// one workgroup.)  With both operands by rows tiles
// go from memory to LDS directly.  Transposing reads are not told apart from such
// loads by the compiler, which waits for all of them before the first read; with
// those a tile goes through registers, one tile further ahead.
//
// WHOLE: for products whose workgroups do not fill the GPU.  With a workgroup or less
// a CU nothing hides the latency of LDS, so the fragments of a whole tile are read
// during the step before (a step of 128 x 128 x 64 took 1400 cycles for 512 of
// products, however many tiles were on their way), and with both operands by rows
// kAhead tiles are on their way.
//
// ANY: operands whose rows are not whole 16-byte chunks, through registers.
template <typename T, typename S, bool A_ROWS, bool B_ROWS, int TA, int TB, int WA, int WB,
          bool WHOLE, bool ANY>
__global__ __launch_bounds__(64 * WA * WB, 2) void product_kernel(ProductArgs p) {
    constexpr int waves = WA * WB, ca = TA / WA, rb = TB / WB, na = ca / 32, nb = rb / 32;
    constexpr bool direct = A_ROWS && B_ROWS && !ANY;
    using A = Operand<T, A_ROWS, TA, waves>;
    using B = Operand<T, B_ROWS, TB, waves>;
    constexpr int bytes = A::kBytes + B::kBytes;
    extern __shared__ __align__(16) char lds[];
    const int wave = wave_id(), lane = lane_id();
    const int wa = wave % WA, wb = wave / WA;
    uint32_t ta, tb, split;
    tile_of(p, ta, tb, split);
    const int64_t a0 = (int64_t)ta * TA, b0 = (int64_t)tb * TB;
    const int32_t first = (int32_t)((int64_t)p.steps * split / p.splits);
    const int32_t last = (int32_t)((int64_t)p.steps * (split + 1) / p.splits);
    const A as(p.a, a0, p.out.cols, wave, lane);
    const B bs(p.b, b0, p.out.rows, wave, lane);
    f32x16 acc[na][nb];
#pragma unroll
    for (int i = 0; i < na; ++i)
#pragma unroll
        for (int j = 0; j < nb; ++j) acc[i][j] = f32x16{};
    constexpr int kcs = kDeep / 16, pieces = A::kPer + B::kPer;
    constexpr int parts = WHOLE ? kcs : 1, places = WHOLE && direct ? kAhead : 2;
    typename Mma<T>::x8 af[2][parts][na], bf[2][parts][nb];
    // fragment x of a part's operands, the rows' first
    auto read = [&](int x, int to, const char* tile, int kc) {
        const int part = WHOLE ? kc : 0;
        if (x < nb)
            bf[to][part][x] = B::template frag<false>(tile + A::kBytes, wb * rb + 32 * x, kc, lane);
        else
            af[to][part][x - nb] = A::template frag<true>(tile, wa * ca + 32 * (x - nb), kc, lane);
    };
    u32x4 held[direct ? 1 : pieces];
    __amdgpu_buffer_rsrc_t ar, br;
    uint32_t ao = 0, bo = 0;
    int64_t aimed = 0;
    bool second = false;
    // of ANY, past the rows' ends: in the tile that is fetched and the one before it
    int32_t a_over[2] = {}, b_over[2] = {};
    auto aim = [&](int32_t step) {
        second = step >= p.half;
        aimed = (int64_t)(second ? step - p.half : step) * kDeep;
        if constexpr (ANY) {
            a_over[1] = a_over[0];
            b_over[1] = b_over[0];
            a_over[0] = as.over_of(aimed);
            b_over[0] = bs.over_of(aimed);
            return;
        }
        ar = as.buffer(aimed, second, p.depth, ao);
        br = bs.buffer(aimed, second, p.depth, bo);
    };
    // piece x of the tile that was aimed at
    auto start = [&](int x, char* tile) {
        if constexpr (direct) {
            if (x < A::kPer) as.load(tile, x, ar, ao, wave);
            else bs.load(tile + A::kBytes, x - A::kPer, br, bo, wave);
        } else if constexpr (ANY) {
            held[x] = x < A::kPer ? as.fetch_any(x, aimed, second, p.depth, a_over[0])
                                  : bs.fetch_any(x - A::kPer, aimed, second, p.depth, b_over[0]);
        } else {
            held[x] = x < A::kPer ? as.fetch(x, ar, ao) : bs.fetch(x - A::kPer, br, bo);
        }
    };
    // and into LDS, of the tile aimed at `ago` aims before
    auto finish = [&](int x, char* tile, int ago) {
        if constexpr (ANY)
            held[x] = x < A::kPer ? A::moved(held[x], a_over[ago]) : B::moved(held[x], b_over[ago]);
        if constexpr (!direct) {
            if (x < A::kPer) A::put(tile, x, held[x], wave, lane);
            else B::put(tile + A::kBytes, x - A::kPer, held[x], wave, lane);
        }
    };
    auto place = [&](int at) { return lds + at * bytes; };
    if constexpr (WHOLE) {
        constexpr int reads = kcs * (na + nb), products = kcs * na * nb;
        if (first < last) {
            // past the end zeros come
#pragma unroll
            for (int t = 0; t < places; ++t) {
                aim(first + t);
#pragma unroll
                for (int x = 0; x < pieces; ++x) start(x, place(t));
#pragma unroll
                for (int x = 0; x < pieces; ++x) finish(x, place(t), 0);
            }
            if constexpr (direct) {
                step_barrier<(places - 1) * pieces>();
            } else {
                aim(first + 2);
#pragma unroll
                for (int x = 0; x < pieces; ++x) start(x, place(0));
                __syncthreads();
            }
            int at = 0, next = 1;
#pragma unroll
            for (int x = 0; x < reads; ++x) read(x % (na + nb), 0, place(0), x / (na + nb));
            auto step = [&](auto parity, int32_t s) {
                constexpr int now = decltype(parity)::value;
                // the next tile is there, and this one is read
                if constexpr (direct) step_barrier<(places - 2) * pieces>();
                else step_barrier<63>();
                aim(s + (direct ? places : 3));
                char* from = place(next);
                char* to = place(at);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int m = 0; m < products; ++m) {
                    const int kc = m / (na * nb), i = m / nb % na, j = m % nb;
                    acc[i][j] = Mma<T>::mul(af[now][kc][i], bf[now][kc][j], acc[i][j]);
                    // the reads in the first half, so that they are there in time
#pragma unroll
                    for (int x = 0; x < reads; ++x)
                        if (x * (products / 2) / reads == m)
                            read(x % (na + nb), now ^ 1, from, x / (na + nb));
#pragma unroll
                    for (int x = 0; x < pieces; ++x)
                        if (x * products / pieces == m) {
                            finish(x, to, 1);
                            start(x, to);
                        }
                    __builtin_amdgcn_sched_barrier(0);
                }
                at = next;
                next = next + 1 < places ? next + 1 : 0;
            };
            int32_t s = first;
            for (; s + 1 < last; s += 2) {
                step(std::integral_constant<int, 0>{}, s);
                step(std::integral_constant<int, 1>{}, s + 1);
            }
            if (s < last) step(std::integral_constant<int, 0>{}, s);
            step_barrier<0>();  // nothing is under way to the tiles, and they are read
        }
    } else if (first < last) {
        constexpr int early = pieces / 2;
        if constexpr (direct) {
            // past the end zeros come
#pragma unroll
            for (int t = 0; t + 1 < places; ++t) {
                aim(first + t);
#pragma unroll
                for (int x = 0; x < pieces; ++x) start(x, place(t));
            }
            step_barrier<(places - 2) * pieces>();
            aim(first + places - 1);
#pragma unroll
            for (int x = 0; x < early; ++x) start(x, place(places - 1));
        } else {
            aim(first);
#pragma unroll
            for (int x = 0; x < pieces; ++x) start(x, place(0));
#pragma unroll
            for (int x = 0; x < pieces; ++x) finish(x, place(0), 0);
            aim(first + 1);
#pragma unroll
            for (int x = 0; x < pieces; ++x) start(x, place(1));
#pragma unroll
            for (int x = 0; x < early; ++x) finish(x, place(1), 0);
            aim(first + 2);
#pragma unroll
            for (int x = 0; x < early; ++x) start(x, place(1));
            __syncthreads();
        }
        int at = 0, next = 1, before = places - 1;  // places of this tile and its neighbours
#pragma unroll
        for (int x = 0; x < na + nb; ++x) read(x, 0, place(at), 0);
        for (int32_t s = first; s < last; ++s) {
#pragma unroll
            for (int kc = 0; kc < kcs; ++kc) {
                const bool end = kc + 1 == kcs;
                if (end) {
                    // the next tile is there, and this one is read
                    if (direct) step_barrier<(places - 2) * pieces>();
                    else __syncthreads();
                    aim(s + (direct ? places : 3));
                }
                char* from = place(end ? next : at);
                char* to = place(end ? at : before);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < na; ++i) {
#pragma unroll
                    for (int j = 0; j < nb; ++j)
                        acc[i][j] = Mma<T>::mul(af[kc & 1][0][i], bf[kc & 1][0][j], acc[i][j]);
                    // between the products what later ones need: fragments of
                    // the next 16 k, and pieces of the tile that takes the place
                    // of the one read last
#pragma unroll
                    for (int x = 0; x < na + nb; ++x)
                        if (x * na / (na + nb) == i) read(x, (kc + 1) & 1, from, end ? 0 : kc + 1);
#pragma unroll
                    for (int x = 0; x < pieces; ++x)
                        if ((end && x < early && x * na / early == i) ||
                            (kc == 0 && x >= early && (x - early) * na / (pieces - early) == i)) {
                            finish(x, to, 1);
                            start(x, to);
                        }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            before = at;
            at = next;
            next = next + 1 < places ? next + 1 : 0;
        }
        step_barrier<0>();  // nothing is under way to the tiles, and they are read
    }

    // The result through LDS, 32 rows of the wave's at a time, so that a row's
    // columns leave side by side.
    constexpr int pitch = out_pitch<ca>(), lanes = ca / 8, at_once = 64 / lanes;
    float* stage = reinterpret_cast<float*>(lds) + wave * (32 * pitch);
    const int64_t c = a0 + wa * ca + 8 * (lane % lanes);
    float bias[8];
    load_bias<T>(bias, p.out, p.parts ? p.out.cols : c);
#pragma unroll
    for (int j = 0; j < nb; ++j) {
        wave_fence();
#pragma unroll
        for (int i = 0; i < na; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float* to = stage + (lane & 31) * pitch + 32 * i + 16 * (g >> 1) +
                            8 * (lane >> 5) + 4 * (g & 1);
                *reinterpret_cast<f4*>(to) = f4{acc[i][j][4 * g], acc[i][j][4 * g + 1],
                                                acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
            }
        wave_fence();
        const int64_t r0 = b0 + wb * rb + 32 * j;
        const int32_t left = (int32_t)(p.out.rows - r0 < 32 ? p.out.rows - r0 : 32);
        if (c >= p.out.cols) continue;
        const float* from = stage + 8 * (lane % lanes);
        if (p.parts) {
            float* to = p.parts + ((int64_t)split * p.out.rows + r0) * p.padded + c;
            for (int r = lane / lanes; r < left; r += at_once) {
                *reinterpret_cast<f4*>(to + r * p.padded) =
                    *reinterpret_cast<const f4*>(from + r * pitch);
                *reinterpret_cast<f4*>(to + r * p.padded + 4) =
                    *reinterpret_cast<const f4*>(from + r * pitch + 4);
            }
            continue;
        }
        with_act(p.out.act, [&](auto act) {
#pragma unroll 2
            for (int r = lane / lanes; r < left; r += at_once) {
                const f4 lo = *reinterpret_cast<const f4*>(from + r * pitch);
                const f4 hi = *reinterpret_cast<const f4*>(from + r * pitch + 4);
                float z[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                emit8<act.value, S>(p.out, r0 + r, c, bias, z);
            }
        });
    }
}

// Adds the parts of a divided sum in their order and finishes.
template <typename T, typename S>
__global__ __launch_bounds__(kThreads) void product_join_kernel(ProductArgs p) {
    const int64_t groups = p.padded / 8;
    const int64_t all = p.out.rows * groups, step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < all; i += step) {
        const int64_t r = i / groups, c = (i % groups) * 8;
        float z[8] = {};
        for (int32_t s = 0; s < p.splits; ++s) {
            const float* from = p.parts + ((int64_t)s * p.out.rows + r) * p.padded + c;
            const f4 lo = *reinterpret_cast<const f4*>(from);
            const f4 hi = *reinterpret_cast<const f4*>(from + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                z[e] += lo[e];
                z[4 + e] += hi[e];
            }
        }
        float b[8];
        load_bias<T>(b, p.out, c);
        with_act(p.out.act, [&](auto act) { emit8<act.value, S>(p.out, r, c, b, z); });
    }
}

// ---------------------------------------------------------------- few rows
// With few rows the time is that of reading the columns' operand (the weights)
// once.  A workgroup has 16 columns and all rows; its waves share the sum, each
// reading its part of the weights' rows straight into the operands of 16 x 16 x 32
// products, and are joined in LDS.  Rows may lie anywhere: nothing is laid out anew.
// (One token over 8192 x 2048 in a graph of such calls: 8.4 us, 4.0 TB/s with the
// launch; 8 rows over 16384 x 4096: 29 us, 4.6 TB/s.)
template <typename T>
struct Mma16;
template <>
struct Mma16<bf16> {
    static __device__ __forceinline__ f4 mul(Mma<bf16>::x8 a, Mma<bf16>::x8 b, f4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Mma16<f16> {
    static __device__ __forceinline__ f4 mul(Mma<f16>::x8 a, Mma<f16>::x8 b, f4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

template <typename T>
__device__ __forceinline__ typename Mma<T>::x8 load_any(const T* p) {
    typedef u32x4 Any __attribute__((aligned(2)));
    return __builtin_bit_cast(typename Mma<T>::x8, *reinterpret_cast<const Any*>(p));
}

template <typename T>
__device__ __forceinline__ typename Mma<T>::x8 load_end(const T* p, int64_t n) {
    typename Mma<T>::x8 x = {};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) x[e] = p[e];
    return x;
}

// Columns of a workgroup, rows at most (8192 columns over 2048: 16, 32, 48 and 64 rows
// 9.8, 13.5, 17 and 21 us; by tiles 12.6, 14.2, 15.2 and 15.7).
constexpr int kFewCols = 16, kFewRows = 32;

template <typename T, int RB, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void product_few_kernel(ProductArgs p) {
    __shared__ float sums[WAVES][16 * RB][kFewCols + 1];
    using x8 = typename Mma<T>::x8;
    const int wave = wave_id(), lane = lane_id(), i = lane & 15, q = lane >> 4;
    const int64_t c0 = (int64_t)blockIdx.x * kFewCols;
    const int64_t c = c0 + i < p.out.cols ? c0 + i : p.out.cols - 1;  // what is past the last
                                                                       // is not stored
    const T* w = (const T*)p.a.p + c * p.a.ld + 8 * q;
    const T* x[RB];
    bool ok[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        ok[b] = 16 * b + i < p.out.rows;
        x[b] = (const T*)p.b.p + (ok[b] ? 16 * b + i : 0) * p.b.ld + 8 * q;
    }
    const int64_t blocks = (p.depth + 63) / 64, whole = p.depth / 64;
    const int64_t first = blocks * wave / WAVES, last = blocks * (wave + 1) / WAVES;
    const int64_t end = last < whole ? last : whole;
    f4 acc[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) acc[b] = f4{};
    int64_t t = first;
    constexpr int kAtOnce = 4;  // blocks of 64 k (eight: one token over 8192 x 2048 8.6 us for 8.4)
    for (; t + kAtOnce <= end; t += kAtOnce) {
        x8 wf[2 * kAtOnce], xf[RB][2 * kAtOnce];
#pragma unroll
        for (int u = 0; u < 2 * kAtOnce; ++u)
            wf[u] = load_any(w + 64 * (t + u / 2) + 32 * (u & 1));
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int u = 0; u < 2 * kAtOnce; ++u)
                xf[b][u] = ok[b] ? load_any(x[b] + 64 * (t + u / 2) + 32 * (u & 1)) : x8{};
#pragma unroll
        for (int u = 0; u < 2 * kAtOnce; ++u)
#pragma unroll
            for (int b = 0; b < RB; ++b) acc[b] = Mma16<T>::mul(wf[u], xf[b][u], acc[b]);
    }
    for (; t < last; ++t) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t k = 64 * t + 32 * h, n = p.depth - k - 8 * q;
            const x8 wf = n >= 8 ? load_any(w + k) : load_end(w + k, n);
#pragma unroll
            for (int b = 0; b < RB; ++b) {
                x8 xf = {};
                if (ok[b]) xf = n >= 8 ? load_any(x[b] + k) : load_end(x[b] + k, n);
                acc[b] = Mma16<T>::mul(wf, xf, acc[b]);
            }
        }
    }
    // a lane has columns 4 q ... + 3 of row i
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[wave][16 * b + i][4 * q + e] = acc[b][e];
    __syncthreads();
    const ProductOut& o = p.out;
    for (int at = threadIdx.x; at < 16 * RB * kFewCols; at += 64 * WAVES) {
        const int r = at / kFewCols, k = at % kFewCols;
        const int64_t col = c0 + k;
        if (r >= o.rows || col >= o.cols) continue;
        float z = 0.0f;
#pragma unroll
        for (int s = 0; s < WAVES; ++s) z += sums[s][r][k];
        if (o.bias) z += o.bias_wide ? ((const float*)o.bias)[col] : (float)((const T*)o.bias)[col];
        if (o.pre) ((T*)o.pre)[r * o.ld_pre + col] = (T)z;
        with_act(o.act, [&](auto act) { z = activate<act.value>(z); });
        if (o.residual) z += (float)((const T*)o.residual)[r * o.ld_r + col];
        ((T*)o.out)[r * o.ld + col] = (T)z;
    }
}

template <typename T, int RB>
void launch_few_waves(const ProductArgs& p, hipStream_t st) {
    const int64_t groups = (p.out.cols + kFewCols - 1) / kFewCols, blocks = (p.depth + 63) / 64;
    const dim3 grid((unsigned)groups);
    // enough waves for the memory's latency, each with a few blocks of k
    if (groups >= 512 || blocks <= 8)
        hipLaunchKernelGGL((product_few_kernel<T, RB, 4>), grid, dim3(256), 0, st, p);
    else if (groups >= 256 || blocks <= 16)
        hipLaunchKernelGGL((product_few_kernel<T, RB, 8>), grid, dim3(512), 0, st, p);
    else
        hipLaunchKernelGGL((product_few_kernel<T, RB, 16>), grid, dim3(1024), 0, st, p);
}

template <typename T>
void launch_few(const ProductArgs& p, hipStream_t st) {
    if (p.out.rows <= 16) launch_few_waves<T, 1>(p, st);
    else launch_few_waves<T, 2>(p, st);
}

// ---------------------------------------------------------------- operands laid out anew
__global__ __launch_bounds__(kThreads) void pad_rows_kernel(PadRows one, PadRows two) {
    const int64_t first = one.rows * (one.padded / 8);
    const int64_t all = first + two.rows * (two.padded / 8);
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < all;
         i += (int64_t)gridDim.x * kThreads) {
        const PadRows& a = i < first ? one : two;
        const int64_t groups = a.padded / 8, at = i < first ? i : i - first;
        const int64_t r = at / groups, c = (at % groups) * 8;
        const uint16_t* p = (const uint16_t*)a.from + r * a.ld + c;
        u32x4 x = {};
        if (c + 8 <= a.cols) {
            x = *reinterpret_cast<const Words8<uint16_t>::Any*>(p);
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (c + e < a.cols) x[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
        }
        *reinterpret_cast<u32x4*>((uint16_t*)a.to + r * a.padded + c) = x;
    }
}

// ---------------------------------------------------------------- the activation's slope
// d as the sum of two numbers of the element type: to 2^-15 of it (bfloat16), or to
// 2^-21 or 2^-25 absolute (float16; 2^-14 past the type's range, where a slope above 1
// may lead).  The first is cut off below d's magnitude, never d itself, so that both have its
// sign (from 2^-116 and from 2^-23 on) and an infinity in the other operand meets no 0
// and no opposite number.
__device__ __forceinline__ float below(float d) {  // of d >= 0
    const uint32_t u = __float_as_uint(d);
    return __uint_as_float(u - (u ? 1u : 0u));
}
__device__ __forceinline__ void two_parts(float d, bf16& first, bf16& rest) {
    const float cut = below(__builtin_fabsf(d));
    first = __builtin_bit_cast(bf16, (uint16_t)(__float_as_uint(__builtin_copysignf(cut, d)) >> 16));
    rest = (bf16)(d - (float)first);
}
__device__ __forceinline__ void two_parts(float d, f16& first, f16& rest) {
    // the rest is a float16 number above 0, so it is 2^-24 at least
    const float most = __builtin_fabsf(d);
    const float cut = fminf(below(most), fmaxf(most - 0x1p-24f, 0.0f));
    first = (f16)__builtin_amdgcn_cvt_pkrtz(__builtin_copysignf(cut, d), 0.0f)[0];
    rest = (f16)(d - (float)first);
}

// A thread has eight columns of a part of the rows.  8192 x 4096 with a GELU takes 59 us
// with dz in two parts (268 MB, 41 us at a copy's rate) and 47 rounded (201 MB, 31).
// The vector unit is busy half of either time (instructions counted, one a cycle and CU)
// and waves wait two thirds of theirs: bound by the loads under way.
template <typename T, int ACT, bool TWO>
__global__ __launch_bounds__(kThreads) void slope_kernel(SlopeArgs a, int64_t groups,
                                                         int64_t rows_of_part) {
    const int64_t strips = (groups + kThreads - 1) / kThreads;
    const int64_t c = 8 * ((int64_t)(blockIdx.x % strips) * kThreads + threadIdx.x);
    const int64_t part = blockIdx.x / strips, n = a.cols - c;
    if (n <= 0) return;
    const int64_t end = (part + 1) * rows_of_part < a.rows ? (part + 1) * rows_of_part : a.rows;
    float sums[8] = {};
#pragma unroll 8
    for (int64_t r = part * rows_of_part; r < end; ++r) {
        float d[8];
        load_row8(d, (const T*)a.dy + r * a.ld_dy + c, n);
        if (ACT != ONEBIT_NONE) {
            float z[8];
            load_row8(z, (const T*)a.pre + r * a.ld_pre + c, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] *= slope<ACT>(z[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[e] += d[e];
        if (a.dz) {
            // the rest of the last group is zeros
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = e < n ? d[e] : 0.0f;
            T* to = (T*)a.dz + r * a.padded + c;
            if constexpr (TWO) {
                T first[8], rest[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) two_parts(d[e], first[e], rest[e]);
                *reinterpret_cast<u32x4*>(to) = __builtin_bit_cast(u32x4, first);
                *reinterpret_cast<u32x4*>((char*)to + a.rest) = __builtin_bit_cast(u32x4, rest);
            } else {
                store_row8(to, d, 8);
            }
        }
    }
    if (!a.partials) return;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) a.partials[part * a.cols + c + e] = sums[e];
}

template <typename T, typename S, bool A_ROWS, bool B_ROWS, int TA, int TB, int WA, int WB,
          bool WHOLE, bool ANY>
void launch_tile(const ProductArgs& p, hipStream_t st) {
    hipLaunchKernelGGL((product_kernel<T, S, A_ROWS, B_ROWS, TA, TB, WA, WB, WHOLE, ANY>),
                       dim3((unsigned)((int64_t)p.tiles_a * p.tiles_b * p.splits)),
                       dim3(64 * WA * WB),
                       (product_lds<TA, TB, WA, WB>(WHOLE && A_ROWS && B_ROWS && !ANY)), st, p);
}

// (tiles of 64 rows have their operand by rows: product_plan)
template <typename T, typename S, bool A_ROWS, bool B_ROWS, bool ANY>
void launch_small(const ProductArgs& p, const ProductPlan& plan, hipStream_t st) {
    if (plan.tile_b == 64) {
        if constexpr (B_ROWS) launch_tile<T, S, A_ROWS, B_ROWS, 128, 64, 2, 2, true, ANY>(p, st);
    } else if ((int64_t)p.tiles_a * p.tiles_b * p.splits <= kCUs) {
        launch_tile<T, S, A_ROWS, B_ROWS, 128, 128, 2, 4, true, ANY>(p, st);
    } else {
        launch_tile<T, S, A_ROWS, B_ROWS, 128, 128, 2, 2, false, ANY>(p, st);
    }
}

template <typename T, typename S, bool A_ROWS, bool B_ROWS>
void launch_tiles(const ProductArgs& p, const ProductPlan& plan, bool any, hipStream_t st) {
    if (plan.tile_b == 256)
        launch_tile<T, S, A_ROWS, B_ROWS, 256, 256, 2, 4, false, false>(p, st);
    else if (plan.tile_a == 256)
        launch_tile<T, S, A_ROWS, B_ROWS, 256, 128, 4, 2, false, false>(p, st);
    else if (any)
        launch_small<T, S, A_ROWS, B_ROWS, true>(p, plan, st);
    else
        launch_small<T, S, A_ROWS, B_ROWS, false>(p, plan, st);
    if (p.parts) {
        const int64_t groups = (p.out.rows * (p.padded / 8) + kThreads - 1) / kThreads;
        hipLaunchKernelGGL((product_join_kernel<T, S>), dim3((unsigned)(groups < 4096 ? groups : 4096)),
                           dim3(kThreads), 0, st, p);
    }
}

// Binary32 results are those of dw, whose operands both come by their own index.
template <typename T>
void launch_typed(const ProductArgs& p, bool a_rows, bool b_rows, const ProductPlan& plan,
                  bool any, hipStream_t st) {
    if (a_rows) launch_tiles<T, T, true, true>(p, plan, any, st);
    else if (b_rows) launch_tiles<T, T, false, true>(p, plan, any, st);
    else if (p.out.type == ONEBIT_F32) launch_tiles<T, float, false, false>(p, plan, any, st);
    else launch_tiles<T, T, false, false>(p, plan, any, st);
}

int64_t tiles_of(int64_t n, int64_t tile) { return (n + tile - 1) / tile; }

}  // namespace

// The division that a model of the kernels' times takes for the fastest: rounds of
// resident workgroups, each the longer the deeper it is, and the join of parts.
// Microseconds as measured (8192^3: 856, 1043 and 988 with tiles of 256 x 256, 256 x
// 128 and 128 x 128; 4096 x 1024 over 8192: 141, 94 and 77).  Workgroups that do not
// fill the GPU take as long as a CU's loads, 60 bytes a ns: 32 KB a step of 128 x 128,
// 24 KB of 128 x 64 (256 x 1024 over 4096: 40 and 32 us).
ProductPlan product_plan(int64_t rows, int64_t cols, int64_t depth, bool cols_by_rows,
                         bool rows_by_rows) {
    struct Tile {
        int32_t a, b, places;       // places: workgroups at once
        double direct, registers;   // microseconds for one of k, by the tiles' way to LDS
        double half, fixed;         // half: with at most half of the places taken
    };
    static const Tile kinds[] = {{256, 256, 256, 0.0260, 0.0272, 0.0180, 9.0},
                                 {256, 128, 256, 0.0159, 0.0164, 0.0118, 6.0},
                                 {128, 128, 512, 0.0150, 0.0175, 0.0086, 5.0},
                                 {128, 64, 512, 0.0110, 0.0110, 0.0066, 4.5}};
    ProductPlan best = {};
    double least = 0.0;
    const int64_t steps = tiles_of(depth, kDeep);
    for (const Tile& t : kinds) {
        if (t.b == 64 && !rows_by_rows) continue;
        const int64_t tiles = tiles_of(rows, t.b) * tiles_of(cols, t.a);
        for (int64_t splits = 1; splits <= 32; ++splits) {
            if (splits > 1 && (tiles * splits > t.places || splits * 4 > steps)) break;
            const int64_t rounds = tiles_of(tiles * splits, t.places);
            const double per_k = tiles * splits * 2 <= t.places ? t.half
                                 : cols_by_rows                 ? t.direct
                                                                : t.registers;
            const double deep = (double)tiles_of(steps, splits) * kDeep;
            // the parts are written and read at 4 bytes per ns and GPU
            const double join =
                splits > 1 ? 4.0 + (double)(2 * splits * rows * cols * 4) / 4.0e6 : 0.0;
            const double time = (double)rounds * (deep * per_k + t.fixed) + join;
            if (best.splits == 0 || time < least) {
                least = time;
                best.tile_a = t.a;
                best.tile_b = t.b;
                best.splits = (int32_t)splits;
            }
        }
    }
    best.bytes = best.splits > 1
                     ? (size_t)best.splits * rows * ((cols + 7) / 8 * 8) * sizeof(float)
                     : 0;
    return best;
}

int64_t product_depth(int64_t depth, bool two) {
    return two ? 2 * tiles_of(depth, kDeep) * kDeep : depth;
}

bool product_any(const ProductPlan& plan) { return plan.tile_a == 128; }

bool product_few(int64_t rows) { return rows <= kFewRows; }

hipError_t launch_product_few(int32_t dtype, const ProductIn& cols_in, const ProductIn& rows_in,
                              int64_t depth, const ProductOut& out, hipStream_t st) {
    if (out.rows == 0 || out.cols == 0) return hipSuccess;
    ProductArgs p = {};
    p.a = cols_in;
    p.b = rows_in;
    p.out = out;
    p.depth = depth;
    if (dtype == ONEBIT_BF16) launch_few<bf16>(p, st);
    else launch_few<f16>(p, st);
    return hipGetLastError();
}

hipError_t launch_product(int32_t dtype, const ProductIn& cols_in, bool cols_by_rows,
                          const ProductIn& rows_in, bool rows_by_rows, int64_t depth,
                          const ProductOut& out, bool any, float* parts, hipStream_t st) {
    if (out.rows == 0 || out.cols == 0) return hipSuccess;
    // what past_end() needs
    if (any && depth > 0 && (cols_in.row < 8 || rows_in.row < 8)) return hipErrorInvalidValue;
    const bool two = cols_in.rest || rows_in.rest;
    const ProductPlan plan =
        product_plan(out.rows, out.cols, product_depth(depth, two), cols_by_rows, rows_by_rows);
    ProductArgs p = {};
    p.a = cols_in;
    p.b = rows_in;
    p.out = out;
    p.parts = plan.splits > 1 ? parts : nullptr;
    p.depth = depth;
    p.half = two ? (int32_t)tiles_of(depth, kDeep) : INT32_MAX;
    p.steps = (int32_t)tiles_of(product_depth(depth, two), kDeep);
    p.padded = (out.cols + 7) / 8 * 8;
    p.tiles_a = (int32_t)tiles_of(out.cols, plan.tile_a);
    p.tiles_b = (int32_t)tiles_of(out.rows, plan.tile_b);
    p.splits = plan.splits;
    if (dtype == ONEBIT_BF16) launch_typed<bf16>(p, cols_by_rows, rows_by_rows, plan, any, st);
    else launch_typed<f16>(p, cols_by_rows, rows_by_rows, plan, any, st);
    return hipGetLastError();
}

hipError_t launch_pad_rows(const PadRows& one, const PadRows& two, hipStream_t st) {
    const int64_t all = one.rows * (one.padded / 8) + two.rows * (two.padded / 8);
    const int64_t groups = tiles_of(all, kThreads);
    if (groups == 0) return hipSuccess;
    hipLaunchKernelGGL(pad_rows_kernel, dim3((unsigned)(groups < 8192 ? groups : 8192)),
                       dim3(kThreads), 0, st, one, two);
    return hipGetLastError();
}

int64_t slope_parts(int64_t rows, int64_t cols) {
    const int64_t strips = tiles_of(tiles_of(cols, 8), kThreads);
    // the parts' column sums are joined, so few parts, and about four workgroups a CU:
    // the backward pass of 8192 x 4096 x 1024 with a GELU, dz rounded, 207 us, 210 with 2048
    // workgroups and half the rows read ahead, 223 with 4096
    int64_t parts = strips > 0 ? 1024 / strips : 1;
    if (parts > tiles_of(rows, 4)) parts = tiles_of(rows, 4);
    return parts < 1 ? 1 : parts;
}

hipError_t launch_slope(const SlopeArgs& a, hipStream_t st) {
    const int64_t groups = tiles_of(a.cols, 8), strips = tiles_of(groups, kThreads);
    const int64_t parts = slope_parts(a.rows, a.cols);
    const dim3 grid((unsigned)(strips * parts)), block(kThreads);
    const int64_t rows_of_part = tiles_of(a.rows, parts);
    auto launch = [&](auto act, auto two) {
        if (a.dtype == ONEBIT_BF16)
            hipLaunchKernelGGL((slope_kernel<bf16, act.value, two.value>), grid, block, 0, st, a,
                               groups, rows_of_part);
        else
            hipLaunchKernelGGL((slope_kernel<f16, act.value, two.value>), grid, block, 0, st, a,
                               groups, rows_of_part);
    };
    with_act(a.act, [&](auto act) {
        if constexpr (!slope_exact(act.value)) {
            if (a.dz && a.rest) return launch(act, std::true_type{});
        }
        launch(act, std::false_type{});
    });
    return hipGetLastError();
}

}  // namespace onebit
