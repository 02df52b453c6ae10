// Attention of drafted trees over the 4-bit paged cache where many query rows
// (nodes x heads that share a kv head) meet the same keys: the formulas and the
// roundings of attn_kv4.hip,
//   q . K[t]  = sk (sum_d q uk) + mk (sum_d q)
//   sum_t p V = sum_t (p sv) (uv - 8) + sum_t p (mv + 8 sv)
// with the codes decoded once for all rows of a workgroup.
//
// A workgroup of W wavefronts takes 16 W rows, 16 a wavefront, and walks 64 keys
// a step.  Its threads load the next step's codes while this one is computed,
// and write them to LDS as fp16 operands of 16 x 16 x 32 products:
//   K    a row of D channels a key, the codes' bits as subnormal numbers; a
//        dword's eight channels lie as 0 4 1 5 2 6 3 7, the queries alike;
//   V^T  a row of 64 keys a channel, the integers u - 8; channel CH u + e (CH
//        channels of a unit of the page) is row 16 e + u, and a row's keys lie
//        in the order in which the first product leaves them in a lane.
// S^T = K Q^T leaves a query row in four lanes, so that its maximum and sums are
// one value a lane and p goes to the second product, O^T = V^T P^T, in registers.
// Pieces of 16 bytes are permuted within their rows (by the row's number) so that
// the 16 lanes of a cycle meet all banks.
//
// Per key and row the vector ALUs have 10.5 issue slots (the two-term fix-up 2,
// maximum 0.5, exponent 1 + 4, both sums 2, weight with its rounding 1), the matrix
// cores 4 D operations (an fp16 output's two-part weights: 2 slots and 2 D more).
// 8 trees of 64 nodes x 4 heads a kv head before 8192 keys, D = 128, bf16: 124 us
// and 8.6 for the join, of which the ALUs work for 63 %, LDS for 45 % and the
// matrix cores for 27 % (554 TFLOP/s): no unit is at its limit, but all wavefronts
// of a workgroup meet at a barrier every 64 keys.  Four wavefronts a SIMD of 16
// rows, 128 registers each (at D = 128 with 1 to 4 more that are spilled),
// are as fast at D = 128 as two of 32 rows with half the reads of LDS, and faster
// at D = 64 (4 x 64 nodes of 8000 keys: 45 against 51 us).
//
// p sv enters the second product as one fp16 number where the output is bf16, as
// two where it is fp16.  One is off by up to 2^-12 of itself, an eighth of what
// rounding the output is: 16 trees of 32 nodes before up to 8192 keys, a tenth of
// the outputs are the neighbouring bf16 number and the error against 64 bits is
// 0.00167 of the output's norm, 0.00166 with fp32 products and the same rounding at
// the end.  Two would take a fifth longer (107 us a call against 131; 8 x 64 of
// 8192 116 against 140, D = 64 85 against 105).
#include "attn_kv4.h"

namespace bq {
namespace {

typedef unsigned long long u64;

constexpr int kKeys = 64;  // of a step

// f over the four lanes of a row.
template <typename F>
__device__ __forceinline__ float row_lanes(float x, F f)
{
    x = f(x, __shfl_xor(x, 16, 64));
    return f(x, __shfl_xor(x, 32, 64));
}
__device__ __forceinline__ float larger(float x, float y) { return fmaxf(x, y); }
__device__ __forceinline__ float sum_of(float x, float y) { return x + y; }

// Two fp16 integers u - 8 from the codes at bits 0..3 (high: 4..7) of each half;
// bias is 0x64006400 in a register (attn_kv4.hip).
__device__ __forceinline__ uint32_t centred2(bool high, uint32_t w, uint32_t bias)
{
    const h2 x = __builtin_bit_cast(h2, (w & (high ? 0x00f000f0u : 0x000f000fu)) | bias);
    const h2 s = {(_Float16)0.0625f, (_Float16)0.0625f}, c = {(_Float16)-72.0f, (_Float16)-72.0f};
    const h2 b = {(_Float16)-1032.0f, (_Float16)-1032.0f};
    return __builtin_bit_cast(uint32_t, high ? __builtin_elementwise_fma(x, s, c) : x + b);
}

// Byte of 16-byte piece c of row r in LDS, of rows of D channels or of 64 keys.
// Pieces are exclusive-ored with bits of their row, so that piece c ^ x of a row
// is 16 x away by an exclusive or.
template <int D>
__device__ __forceinline__ int k_piece(int r, int c)
{
    return D == 64 ? r * 128 + (c ^ (r >> 1 & 7)) * 16 : r * (2 * D) + (c ^ (r & 15)) * 16;
}
__device__ __forceinline__ int v_piece(int r, int c) { return r * 128 + (c ^ (r >> 1 & 7)) * 16; }

// What the keys of a step have beside their codes.  Two of them lie one behind
// the other, read and written in 8 and 16 bytes.
struct alignas(16) Params {
    uint32_t there[2], bad[2];  // a bit a key: in the cache; V's parameters are no numbers
    uint32_t k[kKeys];          // sk, mk
    float mv[kKeys];            // mv + 8 sv
    uint16_t sv[kKeys];
    int top;                    // the greatest |sv|, its bits
};
static_assert(sizeof(Params) % 16 == 0 && offsetof(Params, there) % 16 == 0 && offsetof(Params, bad) % 8 == 0 &&
                  offsetof(Params, k) % 16 == 0 && offsetof(Params, mv) % 16 == 0 && offsetof(Params, sv) % 8 == 0,
              "vectors of 8 and 16 bytes");

// Sequence b's nodes and keys: all its rows have the same.
__device__ __forceinline__ Rows tree_rows(const AttnKv4Args &p, int b)
{
    Rows r;
    const QueryRows q = query_rows(p, b);
    const int len = min(max(p.seq_lens[b], 0), p.max_blocks << p.page_shift);
    r.q0 = q.first;
    r.rows = q.count * p.group;
    r.base = len - q.len;
    r.pos_min = r.base - 1;
    r.pos_max = min(len, r.base + 32 * p.mask_words) - 1;
    r.lo = p.window > 0 ? max(0, r.base - p.window) & ~(kTile - 1) : 0;
    r.hi = max(r.pos_max + 1, r.lo);
    r.chunk = r.hi - r.lo;
    return r;
}

// A unit of work: a sequence, or a part of its keys.  The units of a split call,
// p.nsplit for each kv head and row tile, are shared out over the sequences by
// their keys: all take the same multiple of 64 keys, the least one with which the
// units suffice (to 1.5 %), so that workgroups last equally long also where
// lengths differ (16 trees of 32 nodes before 2 to 8192 keys, D = 128: 109 us,
// with as many parts for each sequence 126; 3 of 61 before up to 30001 122
// against 154).  A call with no more units than sequences is not split: it lasts
// as long as its longest sequence (40 trees of 64 nodes x 4 heads, one before 30000
// keys and the others before 300: 1256 us).
struct Unit {
    int b;         // sequence, -1: none
    int first, n;  // its units
    uint32_t chunk;
};
__device__ __forceinline__ Unit unit_of(const AttnKv4Args &p, int unit)
{
    if (p.nsplit == 1)
        return {unit, unit, 1, 0x80000000u};
    const int lane = threadIdx.x & 63;
    auto keys_of = [&](int i) {  // -1: no rows
        if (i >= p.batch)
            return -1;
        const Rows r = tree_rows(p, i);
        return r.rows > 0 ? r.chunk : -1;
    };
    auto units_of = [](int keys, uint32_t chunk) { return keys < 0 ? 0 : max(1, (int)(((uint32_t)keys + chunk - 1) / chunk)); };
    const int mine = keys_of(lane);
    float all = (float)max(mine, 0);
    int most = mine;
    for (int i = 64 + lane; i < p.batch; i += 64) {
        const int k = keys_of(i);
        all += (float)max(k, 0);
        most = max(most, k);
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        all += __shfl_xor(all, off, 64);
        most = max(most, __shfl_xor(most, off, 64));
    }
    // Multiples of 64 keys: `high` is enough (n_i <= k_i / chunk + 1, so that
    // sum k_i / (units - sequences) always is), `low` is not, or is 0.
    int low = (int)(all * 0.999f / (float)p.nsplit / kKeys) - 1, high = max(1, ((most - 1) >> 6) + 1);
    if (p.nsplit > p.batch)
        high = min(high, (int)(all * 1.001f / (float)(p.nsplit - p.batch) / kKeys) + 1);
    low = max(low, 0);
    while (high - low > 1 + (high >> 6)) {
        const int mid = (low + high) >> 1;
        int n = units_of(mine, (uint32_t)mid * kKeys);
        for (int i = 64 + lane; i < p.batch; i += 64)
            n += units_of(keys_of(i), (uint32_t)mid * kKeys);
#pragma unroll
        for (int off = 32; off > 0; off >>= 1)
            n += __shfl_xor(n, off, 64);
        if (__builtin_amdgcn_readfirstlane(n) <= p.nsplit)
            high = mid;
        else
            low = mid;
    }
    Unit u = {-1, 0, 0, (uint32_t)high * kKeys};
    int before = 0;
    for (int i = lane; i - lane < p.batch; i += 64) {
        const int n = units_of(i < 64 ? mine : keys_of(i), u.chunk);
        int sum = n;
#pragma unroll
        for (int off = 1; off < 64; off *= 2) {
            const int x = __shfl_up(sum, off, 64);
            sum += lane >= off ? x : 0;
        }
        const int first = before + sum - n;
        const u64 here = __ballot(unit >= first && unit < first + n);
        if (here) {
            const int at = __builtin_ctzll(here);
            u.b = __shfl(i, at, 64);
            u.first = __shfl(first, at, 64);
            u.n = __shfl(n, at, 64);
            break;
        }
        before += __shfl(sum, 63, 64);
    }
    u.b = __builtin_amdgcn_readfirstlane(u.b);
    u.first = __builtin_amdgcn_readfirstlane(u.first);
    u.n = __builtin_amdgcn_readfirstlane(u.n);
    return u;
}

// Where a split call keeps {first, n} of each sequence: behind the parts.
__device__ __forceinline__ int2 *unit_table(const AttnKv4Args &p, int D, int rows)
{
    return (int2 *)(p.part + (int64_t)p.nsplit * p.hkv * p.row_tiles * rows * D);
}

template <typename T, int D, int W>
__global__ __launch_bounds__(64 * W, 4) void attn_tree_kernel(const AttnKv4Args p)
{
    constexpr int ROWS = 16 * W, NT = 64 * W;
    constexpr int kPieces = kKeys * D / 2 / 16;       // of codes of a step, K and V each
    constexpr int kMine = (2 * kPieces + NT - 1) / NT;  // of them a thread's
    constexpr int CH = D / 16;                        // channels of a V unit: 4 or 8
    constexpr int MT = D / 16, KS = D / 32;
    constexpr bool kLow = !T::kBf16;
    constexpr int kBuf = kKeys * D * 2;               // bytes of a step's operands, K and V each: a power of two
    __shared__ __attribute__((aligned(16))) uint8_t lk[2 * kBuf], lv[2 * kBuf];
    __shared__ Params params[2];
    const int tid = threadIdx.x, lane = tid & 63, quad = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int head = blockIdx.x % p.hkv, tile = blockIdx.x / p.hkv % p.row_tiles;
    const Unit unit = unit_of(p, blockIdx.x / p.hkv / p.row_tiles);
    if (unit.b < 0)
        return;
    const int b = unit.b, split = blockIdx.x / p.hkv / p.row_tiles - unit.first;
    if (p.nsplit > 1 && (blockIdx.x % (p.hkv * p.row_tiles) | split | tid) == 0)
        unit_table(p, D, ROWS)[b] = make_int2(unit.first, unit.n);
    const Rows r = tree_rows(p, b);
    if (tile * ROWS >= r.rows)
        return;
    const QueryRows qr = query_rows(p, b);
    const int rows = r.rows;
    const int64_t from = r.lo + (int64_t)split * unit.chunk;
    const int start = (int)min(from, (int64_t)r.hi), end = (int)min(from + unit.chunk, (int64_t)r.hi);

    // Codes of the step, two kinds of pieces: K piece i is 16 bytes of key i / (D / 32),
    // V piece i 16 bytes of the four tokens i / (D / 8) (D = 64: two units, 128: one).
    constexpr int kPerKey = D / 32, kPerFour = D / 8;
    const int *table = p.block_table + (int64_t)b * p.max_blocks;
    const int P = 1 << p.page_shift;
    const int64_t head_bytes = (int64_t)P * (D + 8);
    u4 code[kMine];
    int page[kMine], ppage = 0, slot[kMine];
    uint32_t param = 0;  // a lane a key: K's in the first wavefront, V's in the second
    bool there = false;
    auto is_k = [&](int i) { return tid + i * NT < kPieces; };
    auto key_of = [&](int i) {  // first key of piece i
        const int x = tid + i * NT;
        return is_k(i) ? x / kPerKey : (x - kPieces) / kPerFour * 4;
    };
#pragma unroll
    for (int i = 0; i < kMine; ++i) {  // where it goes
        const int x = tid + i * NT - (is_k(i) ? 0 : kPieces);
        if (is_k(i)) {
            slot[i] = k_piece<D>(x / kPerKey, x % kPerKey * 4);
        } else {
            // group g of four tokens of 32: piece g & 3, its first half for g < 4
            const int g = x / kPerFour;
            slot[i] = v_piece(x % kPerFour * (D == 64 ? 2 : 1), (g >> 3) * 4 + (g & 3)) + (g >> 2 & 1) * 8;
        }
    }
    auto base_of = [&](int page) {
        return p.cache + ((int64_t)((uint32_t)page < (uint32_t)p.num_pages ? page : 0) * p.hkv + head) * head_bytes;
    };
    auto load_pages = [&](int t) {
#pragma unroll
        for (int i = 0; i < kMine; ++i)
            page[i] = table[min(t + key_of(i), end - 1) >> p.page_shift];
        if (wave < 2)
            ppage = table[min(t + lane, end - 1) >> p.page_shift];
    };
    auto load_codes = [&](int t) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int x = tid + i * NT;
            if (2 * kPieces % NT == 0 || x < 2 * kPieces) {
                const int in = min(t + key_of(i), end - 1) & (P - 1);
                const int at = is_k(i) ? in * (D / 2) + x % kPerKey * 16
                                       : ((D / 2) << p.page_shift) + (in & ~3) * (D / 2) + (x - kPieces) % kPerFour * 16;
                code[i] = *(const u4 *)(base_of(page[i]) + at);
            }
        }
        if (wave < 2) {
            there = t + lane < end && (uint32_t)ppage < (uint32_t)p.num_pages;
            param = *(const uint32_t *)(base_of(ppage) + ((D + 4 * wave) << p.page_shift) + (min(t + lane, end - 1) & (P - 1)) * 4);
        }
    };
    uint32_t bias = 0x64006400u;
    asm volatile("" : "+v"(bias));
    // -0 that the compiler does not know: a product with a 16-bit factor then is one
    // mixed multiply-add
    float nothing = -0.0f;
    asm volatile("" : "+v"(nothing));
    auto decode = [&](int buf) {
        const int flip = buf * kBuf;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const u4 c = code[i];
            if (is_k(i)) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *(u4 *)(lk + (flip + (slot[i] ^ 16 * j))) =
                        (u4){c[j] & 0x000f000fu, c[j] >> 4 & 0x000f000fu, c[j] >> 8 & 0x000f000fu, c[j] >> 12 & 0x000f000fu};
            } else if (2 * kPieces % NT == 0 || tid + i * NT < 2 * kPieces) {
                // channel CH unit + e in row 16 e + unit; units 2 j and 2 j + 1 have the same permutation
                if constexpr (D == 64) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int by = e & 2 ? 8 : 0;
                            *(u2 *)(lv + flip + slot[i] + 128 * j + 2048 * e) = (u2){centred2(e & 1, c[2 * j] >> by, bias),
                                                                                     centred2(e & 1, c[2 * j + 1] >> by, bias)};
                        }
                } else {
                    const uint32_t lo0 = pack_lo(c[0], c[1]), lo1 = pack_lo(c[2], c[3]);
                    const uint32_t hi0 = pack_hi(c[0], c[1]), hi1 = pack_hi(c[2], c[3]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t w0 = e < 4 ? lo0 : hi0, w1 = e < 4 ? lo1 : hi1;
                        const int by = e & 2 ? 8 : 0;
                        *(u2 *)(lv + flip + slot[i] + 2048 * e) = (u2){centred2(e & 1, w0 >> by, bias), centred2(e & 1, w1 >> by, bias)};
                    }
                }
            }
        }
        // A key that is not there counts for nothing, one whose parameters are no
        // numbers makes NaN of the scores of the rows that see it.
        if (wave < 2) {
            Params &to = params[buf];
            const bool number = (param & 0x7c00u) != 0x7c00u && (param & 0x7c000000u) != 0x7c000000u;
            const uint32_t v = there && number ? param : 0;
            if (wave == 0) {
                to.k[lane] = there && !number ? 0x7e00u : v;
                const u64 all = __ballot(there);
                if (lane == 0)
                    *(u2 *)to.there = (u2){(uint32_t)all, (uint32_t)(all >> 32)};
            } else {
                const float sv = half_bits(v & 0xffffu);
                to.sv[lane] = (uint16_t)v;
                to.mv[lane] = half_bits(v >> 16) + 8.0f * sv;
                const u64 bad = __ballot(there && !number);
                // the greatest of the wavefront in its last lane; the bits are in the order of the numbers
                int top = __float_as_int(fabsf(sv));
                top = max(top, __builtin_amdgcn_update_dpp(0, top, 0x111, 0xf, 0xf, true));
                top = max(top, __builtin_amdgcn_update_dpp(0, top, 0x112, 0xf, 0xf, true));
                top = max(top, __builtin_amdgcn_update_dpp(0, top, 0x114, 0xf, 0xf, true));
                top = max(top, __builtin_amdgcn_update_dpp(0, top, 0x118, 0xf, 0xf, true));
                top = max(top, __builtin_amdgcn_update_dpp(0, top, 0x142, 0xa, 0xf, false));
                top = max(top, __builtin_amdgcn_update_dpp(0, top, 0x143, 0xc, 0xf, false));
                if (lane == 63) {
                    *(u2 *)to.bad = (u2){(uint32_t)bad, (uint32_t)(bad >> 32)};
                    to.top = top;
                }
            }
        }
    };
    if (start < end)
        load_pages(start);

    // this lane's query row: a quarter of its pieces; computed again where it is
    // needed again, so that nothing of it stays in registers
    auto my_row = [&] {
        int x = tid;
        asm volatile("" : "+v"(x));
        return tile * ROWS + 16 * wave + (x & 15);
    };
    u4 q[KS];
    float a1, b1;
    {
        const int row = min(my_row(), rows - 1), node = row / p.group, hg = row - node * p.group;
        const uint16_t *src = (const uint16_t *)p.q + (int64_t)(qr.first + node) * p.q_stride + (head * p.group + hg) * D;
#pragma unroll
        for (int i = 0; i < KS; ++i)
            q[i] = *(const u4 *)(src + (4 * i + quad) * 8);
        if (start < end) {
            load_codes(start);
            load_pages(min(start + kKeys, end - 1));
        }
        float sum = 0.0f, top = 0.0f;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            if (p.scale < 0.0f)  // the sign goes to the query
                q[i] ^= 0x80008000u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = T::to_f32(q[i][j] & 0xffffu), y = T::to_f32(q[i][j] >> 16);
                sum += x;
                sum += y;
                top = fmaxf(top, fmaxf(fabsf(x), fabsf(y)));
            }
        }
        sum = row_lanes(sum, sum_of);
        top = row_lanes(top, larger);
        float back = 1.0f, f = 1.0f;
        if constexpr (T::kBf16) {
            // a power of two brings the row into fp16's range: bf16's eight bits
            // survive down to 2^-24 of the row's largest value
            const uint32_t e = max((__float_as_uint(top) >> 23) & 255u, 11u);
            f = e < 255u ? __uint_as_float((264u - e) << 23) : 1.0f;
            back = e < 255u ? __uint_as_float((e - 10u) << 23) : 1.0f;
        }
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            u4 w = q[i];
            if constexpr (T::kBf16)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = F16::from_f32(T::to_f32(w[j] & 0xffffu) * f) | (uint32_t)F16::from_f32(T::to_f32(w[j] >> 16) * f) << 16;
            q[i] = (u4){pack_lo(w[0], w[2]), pack_hi(w[0], w[2]), pack_lo(w[1], w[3]), pack_hi(w[1], w[3])};
        }
        a1 = fmaxf(back * 0x1p24f * (fabsf(p.scale) * kLog2e), 0x1p-120f);  // a masked score is -inf a1
        b1 = sum * f * 0x1p-24f;
    }
    const bool busy = tile * ROWS + 16 * wave < rows;
    float mt = kNoMax, mref = kNoMax, l = 0.0f, z = 0.0f, cap = 0.0f;  // as attn_kv4.hip's
    f4 o[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
        o[i] = (f4){0, 0, 0, 0};
    // what this lane reads of LDS: its row of a tile, with the exclusive or of its pieces
    const int rk = k_piece<D>(lane & 15, quad), rv = v_piece(lane & 15, quad);

    if (start < end) {
        decode(0);
        if (start + kKeys < end) {
            load_codes(start + kKeys);
            load_pages(min(start + 2 * kKeys, end - 1));
        }
        __syncthreads();
    }
    int buf = 0;
    for (int t = start; t < end; t += kKeys, buf ^= 1) {
        // the next step's operands, and the loads of the one after it
        if (t > start)
            __syncthreads();
        const Params &par = params[buf];
        const u4 flags = *(const u4 *)par.there;
        const float vtop = __int_as_float(par.top);
        if (t + kKeys < end) {
            decode(buf ^ 1);
            if (t + 2 * kKeys < end) {
                load_codes(t + 2 * kKeys);
                load_pages(min(t + 3 * kKeys, end - 1));
            }
        }
        if (!busy)
            continue;
        const int bk = buf * kBuf + rk, bv = buf * kBuf + rv;
        // keys that are not there, and those that not all rows see
        uint32_t on[2] = {(uint32_t)__builtin_amdgcn_readfirstlane(flags[0]), (uint32_t)__builtin_amdgcn_readfirstlane(flags[1])};
        if ((on[0] & on[1]) != ~0u || t > r.pos_min - 63 || (p.window > 0 && t <= r.pos_max - p.window)) {
            const TreeRow see = tree_row(p, r, qr.len, min(my_row(), rows - 1) / p.group);
#pragma unroll 1
            for (int u = 0; u < 2; ++u) {
                const uint32_t x = (u ? on[1] : on[0]) & see.keys(t + 32 * u, r.base);
                on[0] = u ? on[0] : x;
                on[1] = u ? x : on[1];
            }
        }
        // scores: keys 32 u + 16 h + 4 quad + j
        f4 acc[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                acc[u][h] = (f4){0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    acc[u][h] = F16::mma(*(const u4 *)(lk + 64 * D * u + 32 * D * h + (bk ^ 64 * i)), q[i], acc[u][h]);
        float top = -__builtin_inff();
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u4 k = *(const u4 *)&par.k[32 * u + 16 * h + 4 * quad];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[u][h][j] = __builtin_fmaf(acc[u][h][j], half_bits(k[j] & 0xffffu),
                                                  __builtin_fmaf(half_bits(k[j] >> 16), b1, nothing));
            }
        if (__any((on[0] & on[1]) != ~0u || (flags[2] | flags[3]))) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t mine = on[u] >> 4 * quad, bad = flags[2 + u] >> 4 * quad;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float x = acc[u][i >> 2][i & 3];
                    x = bad >> (16 * (i >> 2) + (i & 3)) & 1 ? __builtin_nanf("") : x;
                    acc[u][i >> 2][i & 3] = mine >> (16 * (i >> 2) + (i & 3)) & 1 ? x : -__builtin_inff();
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
            top = fmaxf(top, acc[i >> 3][i >> 2 & 1][i & 3]);
        if (__builtin_expect(__any(vtop > cap || top * a1 > mt + 8.0f), 0)) {
            // each row by the keys that it sees (attn_kv4.hip)
            float seen = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                seen = fmaxf(seen, acc[i >> 3][i >> 2 & 1][i & 3] > -__builtin_inff()
                                       ? fabsf(half_bits(par.sv[16 * (i >> 2) + 4 * quad + (i & 3)])) : 0.0f);
            top = row_lanes(top, larger);
            seen = row_lanes(seen, larger);
            const bool wider = seen > cap;
            if (wider || top * a1 > mt + 8.0f)
                mt = fmaxf(mt, top * a1);
            // 2 to 4 times the scale
            const uint32_t e = (__float_as_uint(fminf(seen, 65504.0f)) >> 23) + 2u;
            cap = wider ? __uint_as_float(e << 23) : cap;
            const float shift = cap > 0.0f ? 133.0f - (float)(__float_as_uint(cap) >> 23) : 0.0f;
            const float now = mt - shift, f = __builtin_amdgcn_exp2f(mref - now);  // 1 for a row that needs nothing
            mref = now;
            l *= f;
            z *= f;
#pragma unroll
            for (int i = 0; i < MT; ++i)
                o[i] *= f;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            u4 ph, pl;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u2 sv = *(const u2 *)&par.sv[32 * u + 16 * h + 4 * quad];
                const float4 mv = *(const float4 *)&par.mv[32 * u + 16 * h + 4 * quad];
                const float vs[4] = {half_bits(sv[0] & 0xffffu), half_bits(sv[0] >> 16), half_bits(sv[1] & 0xffffu), half_bits(sv[1] >> 16)};
                const float vm[4] = {mv.x, mv.y, mv.z, mv.w};
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    const float p0 = __builtin_amdgcn_exp2f(acc[u][h][j] * a1 - mref);
                    const float p1 = __builtin_amdgcn_exp2f(acc[u][h][j + 1] * a1 - mref);
                    l += p0;
                    l += p1;
                    z += p0 * vm[j];
                    z += p1 * vm[j + 1];
                    const float v0 = __builtin_fmaf(p0, vs[j], nothing), v1 = __builtin_fmaf(p1, vs[j + 1], nothing);
                    const h2 hi = {(_Float16)v0, (_Float16)v1};
                    ph[2 * h + j / 2] = __builtin_bit_cast(uint32_t, hi);
                    if constexpr (kLow)
                        pl[2 * h + j / 2] = __builtin_bit_cast(uint32_t, (h2){(_Float16)(v0 - (float)hi[0]), (_Float16)(v1 - (float)hi[1])});
                }
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const u4 a = *(const u4 *)(lv + 2048 * i + (bv ^ 64 * u));
                o[i] = F16::mma(a, ph, o[i]);
                if constexpr (kLow)
                    o[i] = F16::mma(a, pl, o[i]);
            }
        }
    }
    if (!busy)
        return;
    l = row_lanes(l, sum_of);
    z = row_lanes(z, sum_of);
    const int row = my_row(), node = row / p.group, hg = row - node * p.group;
    if (row >= rows)
        return;
    // lane's channels: unit 4 quad + k has CH of them, register k of tile e
    const int64_t at = (int64_t)(qr.first + node) * p.hq + head * p.group + hg;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t part = (int64_t)blockIdx.x * ROWS + 16 * wave + (lane & 15);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int unit = 4 * quad + k;
        float v[CH];
#pragma unroll
        for (int e = 0; e < CH; ++e)
            v[e] = o[e][k] + z;
        if (p.nsplit == 1) {
            uint32_t y[CH / 2];
#pragma unroll
            for (int e = 0; e < CH; e += 2)
                y[e / 2] = T::from_f32(v[e] * inv) | (uint32_t)T::from_f32(v[e + 1] * inv) << 16;
            uint16_t *dst = (uint16_t *)p.out + at * D + unit * CH;
            if constexpr (CH == 8)
                *(u4 *)dst = (u4){y[0], y[1], y[2], y[3]};
            else
                *(u2 *)dst = (u2){y[0], y[1]};
        } else {
#pragma unroll
            for (int e = 0; e < CH; e += 4)
                *(float4 *)(p.part + part * D + unit * CH + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
    }
    if (quad == 0) {
        if (p.nsplit > 1)
            *(float2 *)(p.part_ml + part * 2) = make_float2(mref, l);
        else if (p.lse)
            p.lse[at] = l == 0.0f ? -__builtin_inff() : (mref + __builtin_amdgcn_logf(l)) * kLn2;
    }
}

// Joins the parts of a query row, D/4 lanes a row.
template <typename T, int D, int ROWS>
__global__ __launch_bounds__(256) void attn_tree_join(const AttnKv4Args p)
{
    constexpr int TEAM = D / 4, MANY = 256 / TEAM;  // rows of a workgroup
    const int per = (p.join_rows + MANY - 1) / MANY;
    const int item = blockIdx.x / per, jr = blockIdx.x % per * MANY + threadIdx.x / TEAM;
    const int head = item % p.hkv, tile = item / p.hkv % p.row_tiles;
    const int b = item / p.hkv / p.row_tiles;
    const QueryRows q = query_rows(p, b);
    const int row = tile * ROWS + jr, c = threadIdx.x % TEAM;
    if (jr >= p.join_rows || row >= q.count * p.group)
        return;
    const int2 units = unit_table(p, D, ROWS)[b];
    const int n = units.y;
    const int64_t step = (int64_t)p.hkv * p.row_tiles * ROWS;  // from a unit's to the next one's
    const int64_t first = units.x * step + (tile * p.hkv + head) * (int64_t)ROWS + jr;
    float mm = kNoMax;
    for (int s = c; s < n; s += TEAM)
        mm = fmaxf(mm, p.part_ml[(first + step * s) * 2]);
#pragma unroll
    for (int off = TEAM / 2; off > 0; off >>= 1)
        mm = fmaxf(mm, __shfl_xor(mm, off, 64));
    float l = 0.0f;
    f4 acc = {0, 0, 0, 0};
#pragma unroll 4
    for (int s = 0; s < n; ++s) {
        const float2 ml = *(const float2 *)(p.part_ml + (first + step * s) * 2);
        const f4 o = *(const f4 *)(p.part + (first + step * s) * D + 4 * c);
        const float f = __builtin_amdgcn_exp2f(ml.x - mm);
        l += f * ml.y;
        acc += f * o;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int qi = row / p.group, hg = row - qi * p.group;
    const int64_t at = (int64_t)(q.first + qi) * p.hq + head * p.group + hg;
    *(u2 *)((uint16_t *)p.out + at * D + 4 * c) = (u2){T::from_f32(acc[0] * inv) | (uint32_t)T::from_f32(acc[1] * inv) << 16,
                                                       T::from_f32(acc[2] * inv) | (uint32_t)T::from_f32(acc[3] * inv) << 16};
    if (p.lse && c == 0)
        p.lse[at] = l == 0.0f ? -__builtin_inff() : (mm + __builtin_amdgcn_logf(l)) * kLn2;
}

template <typename T, int D, int W>
hipError_t launch_t(const AttnKv4Args &p, hipStream_t s)
{
    constexpr int MANY = 1024 / D;
    const int64_t items = (int64_t)p.hkv * p.row_tiles;
    const int64_t groups = items * (p.nsplit > 1 ? p.nsplit : p.batch), joins = p.batch * items * ((p.join_rows + MANY - 1) / MANY);
    if (!grid_fits(groups, 64 * W) || (p.nsplit > 1 && !grid_fits(joins, 256)))
        return kGridTooLarge;
    attn_tree_kernel<T, D, W><<<dim3((unsigned)groups), 64 * W, 0, s>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.nsplit == 1)
        return e;
    attn_tree_join<T, D, 16 * W><<<dim3((unsigned)joins), 256, 0, s>>>(p);
    return hipGetLastError();
}

template <typename T, int D>
hipError_t launch_w(const AttnKv4Args &p, int rt, hipStream_t s)
{
    return rt == 8 ? launch_t<T, D, 8>(p, s) : launch_t<T, D, 16>(p, s);
}

}  // namespace

AttnKv4Plan attn_tree_plan(int64_t batch, int64_t max_q_len, int q_heads, int kv_heads, int D, int64_t max_len)
{
    // max_len is the block table's width, as the lengths are device memory: a table
    // that is wider than its sequences costs the short caches' forms (1 tree of 8 x 4
    // rows, 700 keys 10.1 us, in a table for 32768 14.6; 64 x 4 rows 10.7 and 24.3).
    // Rows times keys from which the operands' way through LDS and the parts of
    // 16 W rows pay: 1 tree of 64 nodes x 4 heads before 8000 keys of 8 kv heads
    // (2^24) 42.6 us against attn_kv4.hip's 37.5, 30000 73.8 and 77.9, 3 x 61 of
    // 8000 67.0 and 81.1, of 30001 173 and 253; D = 64: 8 of 700 31.3 and 22.0, of
    // 2000 (2^25) 38.5 and 35.6, 1 of 128 nodes before 8000 (2^25) 39.7 and 48.8,
    // 8 x 64 of 8192 95 and 115.  D = 256 has no such form: attn_kv4.hip
    // decodes all codes for every 16 rows (8 x 64 of 8192 288 us).
    const int64_t rows = max_q_len * (q_heads / kv_heads);
    if (D > 128 || rows <= 64 || (double)batch * kv_heads * rows * max_len < (D == 128 ? 3 << 24 : 1 << 25)) {
        AttnKv4Plan a = attn_kv4_plan(batch, max_q_len, q_heads, kv_heads, D, max_len);
        // Where 16 rows a workgroup still leave CUs free: they let eight wavefronts
        // have the keys, and no split is needed up to a length (8 kv heads; 1 tree
        // of 8 x 4 rows, 200 keys 7.0 us against 9.7, 700 10.1 against 15.2, 1000
        // 11.6 against 18.0, 1500 13.8 against 13.3 split; 4 of 32 x 4, 1500 17.7
        // against 25.4, 2000 21.3 against 27.3).
        const int64_t tiles = (rows + 15) / 16, items = batch * kv_heads * tiles;
        if (D == 128 && a.rt == 2 && items <= 256 && max_len <= (items >= 128 ? 2048 : 1024)) {
            a.rt = 1;
            a.row_tiles = tiles;
            a.nsplit = 1;
            a.part_rows = 0;
        }
        return a;
    }
    // 256 rows a workgroup, one a CU (16 x 64 nodes x 4 heads before 3000 keys 101
    // us, with 128 rows, two a CU, 108), or 128 where that leaves out a sixth of
    // the rows (130 x 4 rows before 8000 keys 158 us against 200; 275 x 4 161
    // against 152).
    const int64_t few = (rows + 127) / 128 * 128, many = (rows + 255) / 256 * 256;
    AttnKv4Plan a;
    a.rt = few * 6 <= many * 5 ? 8 : 16;
    a.row_tiles = (rows + 16 * a.rt - 1) / (16 * a.rt);
    const int64_t items = kv_heads * a.row_tiles, slots = a.rt == 8 ? 512 : 256;
    // As many units as the CUs hold: each has a prologue and writes its rows'
    // sums (8 x 64 nodes before 8192 keys, in twice as many 149 us against 124).
    const int64_t want = max_len > 1024 ? slots / items : 1, most = batch * ((max_len + 127) / 128);
    const int64_t n = want < most ? want : most;
    a.nsplit = (int)(n > batch ? n : 1);
    // the table of the sequences' units takes rows of its own
    a.part_rows = a.nsplit > 1 ? items * a.nsplit * 16 * a.rt + (2 * batch + D - 1) / D : 0;
    return a;
}

hipError_t launch_attn_tree(AttnKv4Args &p, int D, int rt, bool bf16, hipStream_t s)
{
    if (rt <= 2)
        return launch_attn_kv4(p, D, rt, bf16, s);
    const int64_t rows = (int64_t)p.max_q_len * p.group;
    p.join_rows = (int)(rows < 16 * rt ? rows : 16 * rt);
    if (D == 64)
        return bf16 ? launch_w<BF16, 64>(p, rt, s) : launch_w<F16, 64>(p, rt, s);
    return bf16 ? launch_w<BF16, 128>(p, rt, s) : launch_w<F16, 128>(p, rt, s);
}

}  // namespace bq
