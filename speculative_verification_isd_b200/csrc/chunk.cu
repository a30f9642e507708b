// Attention of a chunk of new tokens per request over the paged cache: the
// prompt's (and plain decoding's) counterpart of the block attention.  Row i
// of request b is the token at position kv_len[b] + i; its K/V row goes to
// its page and it attends to every key at a position <= its own:
//
//   out[i, h] = sum_j 2^(x_ij - m_i) v_j / sum_j 2^(x_ij - m_i),
//   x_ij = sm_scale log2(e) q[i, h] . k_j,   j <= kv_len[b] + i.
//
// One persistent kernel, one CTA per SM, then a small one that joins the
// pieces of work items cut between CTAs:
//
//  * rows are packed: a tile is up to 128 rows (token, head of the KV group),
//    an item is up to two tiles of consecutive tokens of one (request, KV
//    head), so a key tile read once serves 256 rows of a prompt, and every
//    head of a group when decoding;
//  * the items' 128-key tiles, flattened, are cut into one equal range per CTA
//    (the lengths are on the device, so every CTA works the cut out itself);
//  * cached keys come from their pages by TMA, new keys from k_new / v_new
//    themselves, so no product waits for the append.  The softmax warps append a
//    token each at the start, the fixing warp the rest, one by one, while it has
//    nothing to fix and after its last piece.  Behind enough attention that is
//    hidden (55 tokens a CTA in the long prompts below); a call of many new tokens
//    and little attention ends with it (512 prompts of 128 tokens, 443 a CTA: 1.7
//    ms, where its bytes would take 0.25);
//  * S = Q.K^T and O += P.V run on the tensor cores with S, P and O in TMEM
//    (P overwrites S as bf16); a softmax thread owns one row, its maximum and
//    sum live in registers.  Weights are taken by the reference as it stands, an
//    earlier maximum: O is rescaled only when a row has none yet, when half a
//    tile's weights sum to more than 2^10, or, in tiles that some row does not
//    see whole, when the maximum has grown by more than 2^8;
//  * two warpgroups of softmax threads, each with its S and O, so that one's
//    softmax runs under the other's products: in an item of two tiles each
//    has a tile, in an item of one they take the key tiles in turn and add up
//    their O at the end; with at most 32 rows (decoding) the rows are put
//    into Q four times and each warp takes a quarter of a tile's keys;
//  * every wait is bounded (about 2 s): on time-out the CTA raises
//    ISD_FLAG_WAIT_TIMEOUT, all roles leave their loops, copies and MMAs in
//    flight are drained and TMEM is released.
//
// Measured with 32 / 8 heads of 128: four prompts of 2 k tokens behind 4 to 8 k
// (885 GFLOP) 785 to 820 us in one launch, cool, 1.08 to 1.13 PFLOP/s, and 965 call
// after call at the power cap, 0.92; the tensor core and the exponentials' unit
// are at 0.58 to 0.61 each (a tile's scores, weights and product follow one
// another in each of the two warpgroups: 3.3 thousand cycles for 2 x 1024 of
// either).  32 requests of one token behind 512 to 8192 (621 MB) 115 to 120 us,
// 5.2 to 5.4 TB/s, memory; one token behind 1000 tokens 13.5 us and 3.4 for the
// join, nearly all of it latency.
#include <cuda.h>
#include <cuda_runtime.h>

#include "chunk_cut.h"
#include "common.cuh"
#include "launch.h"
#include "plan.h"
#include "sm100.cuh"
#include "tmap.h"

namespace isd {

void set_error_detail(const char* msg);

namespace {

constexpr int kTileRows = 128;          // rows per tile
constexpr int kHalfBytes = kKeys * 128; // 64 dimensions of a K, V or Q tile
// A tile in shared memory is [64-d half][row][128 swizzled bytes].  A cached
// tile whose pages are whole groups of 8 rows is [group][half][row of the
// group][128 bytes] instead: then one box brings a page's rows with both halves
// (a TMA copy takes the producer about 70 cycles to issue).
constexpr int kGroupRows = 8;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kChunkThreads = 384;
constexpr int kLaunchRegs = 168, kRegsLow = 88, kRegsHigh = 208;
static_assert(kRegsLow * 128 + kRegsHigh * 256 <= kLaunchRegs * kChunkThreads, "register split exceeds the launch");

// A cut item, for the joining kernel (written by the CTA with its first keys).
struct ChunkCut {
    int parts;  // CTAs that hold a part, from the writing one on; 0: nothing cut
    int g, i0, i1, start;
    int pad[3];
};

struct ChunkArgs : CutShape {
    int B, T, Hq, Hkv, grp, box, num_pages;
    int tps;        // tokens of a tile of 32 rows
    int grouped;    // layout of a cached tile (see kGroupRows)
    int part_rows;  // rows of a partial result
    float scale_log2;
    const int32_t* page_table;
    const int32_t* kv_len;
    const int32_t* q_start;
    const __nv_bfloat16* k_new;
    const __nv_bfloat16* v_new;
    __nv_bfloat16* k_pool;
    __nv_bfloat16* v_pool;
    __nv_bfloat16* out;
    float* part;    // [grid][2] partials: maxima, sums [part_rows], O [D / 4][part_rows][4]
    ChunkCut* cuts;  // [grid]
    int32_t* err_flag;
};

// This CTA's share of one item, as its roles see it.
enum { kTwo = 0, kOne = 1, kQuad = 2 };
struct Piece {
    int b, g, start, kv, kvt;
    int i0, i1, t0, t1;  // tokens; key tiles (none: no more pieces)
    int mode;            // two row tiles, one, or one of at most 32 rows
    int slot;            // of the partial result, -1 for a whole item
    int merged;          // the new tokens lie in the last cached tile
    int items;           // of the request's KV head
};
constexpr int kPieces = 16;  // pieces that the roles may lie apart

template <int D>
struct ChunkShape {
    static constexpr int kHalves = D / 64;
    static constexpr int kTile = kHalves * kHalfBytes;  // bytes of a Q, K or V tile
    // rings of K and V tiles; a V tile is held longer (until P.V, after its softmax)
    static constexpr int kStagesK = D == 128 ? 2 : 5, kStagesV = D == 128 ? 3 : 5;
    static constexpr int kStages = kStagesK + kStagesV;
    static constexpr int kControl = 3 * 1024;
    static constexpr size_t kSmem() { return (size_t)(2 + kStages) * kTile + kControl; }
};

template <int D>
struct ChunkShared {
    static constexpr int S = ChunkShape<D>::kStages;
    uint64_t full[S], empty[S], fix[S];
    uint64_t q_full[2], q_empty[2];
    // by softmax warpgroup; P in halves of 64 keys, `pv_half` after the first's product
    uint64_t s_full[2], p_full[2][2], pv_half[2], pv_done[2], o_free[2];
    uint64_t meet, drain;
    Piece pieces[kPieces];
    long long my0, total, len, rel;  // the range's start and length; its first item starts at `rel` in it
    int b, g, q;
    Request first;
    uint32_t tmem;
    int abort_flag, never;
    uint32_t published;  // pieces written by the producer
    uint32_t issued[2];  // K, V tiles that their producer has begun to load
    uint32_t appended;   // new tokens taken for appending
    uint32_t fixed;      // pieces that the fixing warp is done with
    uint32_t checked;    // pieces whose `holed` it has set
    uint32_t epilogues[2];  // finished by the warps of a softmax warpgroup (4 a piece)
    int holed[kPieces];  // whether the fixing warp touches every tile of new tokens of a piece
    int bad_piece;       // the piece whose `bad_from` holds, or -1
    int bad_from[3][D];  // first new token with +inf, -inf, NaN in dimension d of V
};

ISD_DEVINL float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// two 32-bit operations at once
ISD_DEVINL unsigned long long pair(float lo, float hi) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
ISD_DEVINL void unpair(unsigned long long v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
ISD_DEVINL unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
ISD_DEVINL unsigned long long add2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

ISD_DEVINL void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
        "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
ISD_DEVINL void tmem_ld32(uint32_t taddr, float (&r)[32]) {
    sm100::tmem_ld_32x32b_x32(taddr, reinterpret_cast<uint32_t(&)[32]>(r));
}
// Waits for the loads so far; the values depend on it, so none is used before.
ISD_DEVINL void tmem_arrived(float (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                   "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]),
                   "+f"(r[15]), "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]),
                   "+f"(r[22]), "+f"(r[23]), "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]));
    asm volatile("" : "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31]));
}
ISD_DEVINL void tmem_ld8(uint32_t taddr, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

// The tensor-core instructions of the MMA warp: the whole warp runs its code and
// one elected lane issues, so that descriptors stay in uniform registers (with a
// branch for lane 0 around the code, an MMA took about 80 cycles to issue, 64
// of the tensor core's).
// (8-row groups 1024 bytes apart, or NH times that in a grouped tile).
constexpr uint32_t kDescHi = 1u << 14 | 2u << 29;  // of smem_desc_sw128, less the groups' distance / 16
ISD_DEVINL void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                       uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b64 da, db;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
        " mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %6};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi | 1024u >> 4), "r"(b_hi)
        : "memory");
}
ISD_DEVINL void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                       uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b64 db;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
        " mov.b64 db, {%2, %5};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(b_hi)
        : "memory");
}
ISD_DEVINL void commit_to(uint64_t* bar) {
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
        : "memory");
}
ISD_DEVINL void mbar_arrive_n(uint64_t* bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;\n" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}

ISD_DEVINL uint64_t policy_evict_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;\n" : "=l"(p));
    return p;
}

ISD_DEVINL void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }

// 32 bytes of a row: a whole sector in one store where the address allows
ISD_DEVINL void store32(void* p, const uint32_t (&r)[8], bool aligned) {
    if (aligned) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                     "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(r[0], r[1], r[2], r[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(r[4], r[5], r[6], r[7]);
    }
}

// Of eight packed bf16, whether one is infinite or NaN: a bit of 0x80008000 is
// set where the exponent is all ones.
ISD_DEVINL uint32_t odd_bits(uint4 w) {
    auto one = [](uint32_t x) { return (x & 0x7fff7fffu) + 0x00800080u; };
    return one(w.x) | one(w.y) | one(w.z) | one(w.w);
}
constexpr uint32_t kOddBits = 0x80008000u;

ISD_DEVINL uint32_t peek(const uint32_t* p) { return *(const volatile uint32_t*)p; }

template <int D>
__global__ void __launch_bounds__(kChunkThreads, 1)
chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_qs,
             const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
             const __grid_constant__ CUtensorMap tm_kn, const __grid_constant__ CUtensorMap tm_vn,
             const __grid_constant__ ChunkArgs a) {
    using namespace sm100;
    using Shape = ChunkShape<D>;
    constexpr int NH = Shape::kHalves, NST = Shape::kStages, NK = Shape::kStagesK, NV = Shape::kStagesV;
    constexpr uint32_t kTmemCols = 512, kTmemO = 256;
    extern __shared__ __align__(1024) unsigned char smem_raw[];  // there is no other shared memory
    unsigned char* sQ = smem_raw;
    unsigned char* ring = sQ + 2 * Shape::kTile;
    ChunkShared<D>* sh = reinterpret_cast<ChunkShared<D>*>(ring + NST * Shape::kTile);
    static_assert(sizeof(ChunkShared<D>) <= Shape::kControl, "control block");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();

    // ---- set-up: barriers, TMEM, and this CTA's range of the work
    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->empty[s], 1);
            mbar_init(&sh->fix[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->q_full[i], 1);
            mbar_init(&sh->q_empty[i], 1);
            mbar_init(&sh->s_full[i], 1);
            mbar_init(&sh->p_full[i][0], 4);
            mbar_init(&sh->p_full[i][1], 4);
            mbar_init(&sh->pv_half[i], 1);
            mbar_init(&sh->pv_done[i], 1);
            mbar_init(&sh->o_free[i], 8);
        }
        mbar_init(&sh->meet, 8);
        mbar_init(&sh->drain, 1);
        sh->abort_flag = sh->never = 0;
        sh->published = sh->issued[0] = sh->issued[1] = sh->appended = sh->fixed = sh->checked = sh->epilogues[0] = sh->epilogues[1] = 0;
        sh->bad_piece = -1;
        sh->b = a.B;
        fence_mbar_init();
    }
    if (warp == 9 && lane == 0) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_qs);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
        prefetch_tmap(&tm_kn);
        prefetch_tmap(&tm_vn);
    }
    if (warp == 8) {
        tmem_alloc(&sh->tmem, kTmemCols);
        tmem_relinquish();
    }
    // what comes before in the stream is done from here on (nothing global was
    // touched so far: the previous call's joining kernel may still read `cuts`)
    pdl_wait();
    if (threadIdx.x == 0) a.cuts[blockIdx.x].parts = 0;
    bool bad = false;
    {
        // costs of the requests, summed in order: a thread per request, and
        // when there are more than threads, once for the total and again up to
        // the request that holds this CTA's first position
        long long* wsum = reinterpret_cast<long long*>(ring);  // 12 warp sums (the ring is not in use yet)
        long long run = 0, before = 0, head = 0;
        Request r = {};
        auto pass = [&](int b) {
            head = 0;
            if (b < a.B) {
                const int s = a.q_start[b], e = a.q_start[b + 1], kv = a.kv_len[b];
                if (s < 0 || e < s || e > a.T) {
                    bad = true;
                } else {
                    r = request_of(a, s, e, kv);
                    head = head_cost(a, r);
                }
            }
            const long long c = head * a.Hkv;
            long long incl = c;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += v;
            }
            __syncthreads();
            if (lane == 31) wsum[warp] = incl;
            __syncthreads();
            before = run + incl - c;
            for (int w = 0; w < kChunkThreads / 32; ++w) {
                if (w < warp) before += wsum[w];
                run += wsum[w];
            }
        };
        for (int b0 = 0; b0 < a.B; b0 += kChunkThreads) pass(b0 + (int)threadIdx.x);
        const long long total = run;
        const int G = cut_ctas(a, total, gridDim.x);
        const bool mine = (int)blockIdx.x < G;
        const long long my0 = mine ? cut_start(total, G, blockIdx.x) : 0;
        const long long my1 = mine ? cut_start(total, G, blockIdx.x + 1) : 0;
        if (threadIdx.x == 0) {
            sh->my0 = my0;
            sh->total = total;
            sh->len = my1 - my0;
        }
        auto locate = [&](int b) {
            if (my0 >= my1 || my0 < before || my0 >= before + head * a.Hkv) return;
            int g, q;
            const int rem = cut_item(a, r, head, my0 - before, g, q);
            sh->b = b;
            sh->g = g;
            sh->q = q;
            sh->rel = -rem;
            sh->first = r;
        };
        if (a.B <= kChunkThreads) {
            locate(threadIdx.x);
        } else {
            run = 0;
            for (int b0 = 0; b0 < a.B; b0 += kChunkThreads) {
                pass(b0 + (int)threadIdx.x);
                locate(b0 + (int)threadIdx.x);
            }
        }
    }
    proxy_fence();
    tc_fence_before();
    bad = __syncthreads_or(bad);
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    if (bad && blockIdx.x == 0 && threadIdx.x == 0) raise_flag(a.err_flag, ISD_FLAG_CHUNK_RANGE);
    volatile int* abort_flag = &sh->abort_flag;
    auto give_up = [&]() {
        *abort_flag = 1;
        raise_flag(a.err_flag, ISD_FLAG_WAIT_TIMEOUT);
    };
    // waits on a counter in shared memory; every lane that asks gets the answer.  The
    // limit runs from the counter's last step: the fixing warp waits for the last
    // tile of a piece from its first on, whose millions of tiles may take seconds.
    auto until = [&](const uint32_t* counter, uint32_t least) {
        uint32_t at = peek(counter);
        if (at >= least) return true;
        uint64_t t_step = global_ns();
        for (uint32_t it = 1; peek(counter) < least; ++it) {
            __nanosleep(20);
            if (it & 63) continue;
            if (const uint32_t now = peek(counter); now != at) {
                at = now;
                t_step = global_ns();
            }
            if (*abort_flag || global_ns() - t_step > kWaitNs) {
                give_up();
                return false;
            }
        }
        return true;
    };
    // Appends one token of this CTA's share of the new rows to its page, 16 bytes
    // a lane; false when all are taken.
    const int t_new = (int)((long long)a.T * blockIdx.x / gridDim.x);
    const int t_end = bad ? t_new : (int)((long long)a.T * (blockIdx.x + 1) / gridDim.x);
    auto append = [&]() {
        int t = 0;
        if (lane == 0) t = t_new + (int)atomicAdd(&sh->appended, 1u);
        t = __shfl_sync(0xffffffffu, t, 0);
        if (t >= t_end) return false;
        int b = -1;  // the last request that starts at or before t
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const uint32_t at = __ballot_sync(0xffffffffu, b0 + lane < a.B && a.q_start[b0 + lane] <= t);
            b += __popc(at);
            if (at != 0xffffffffu) break;
        }
        if (b < 0 || t >= a.q_start[b + 1]) return true;  // a row of no request
        const int start = a.q_start[b], kv = a.kv_len[b];
        if (chunk_tokens(a, kv, a.q_start[b + 1] - start) == 0) {
            if (lane == 0) raise_flag(a.err_flag, ISD_FLAG_CAPACITY);
            uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)t * a.Hq * D);
            for (int i = lane; i < a.Hq * D / 8; i += 32) o[i] = make_uint4(0, 0, 0, 0);
            return true;
        }
        const int at = kv + (t - start);
        const int page = a.page_table[(size_t)b * a.max_pages + at / a.P];
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0) raise_flag(a.err_flag, ISD_FLAG_PAGE_OOB);
            return true;
        }
        const size_t dst = ((size_t)page * a.P + at % a.P) * a.Hkv * D, src = (size_t)t * a.Hkv * D;
        const uint4* ks = reinterpret_cast<const uint4*>(a.k_new + src);
        const uint4* vs = reinterpret_cast<const uint4*>(a.v_new + src);
        uint4* kd = reinterpret_cast<uint4*>(a.k_pool + dst);
        uint4* vd = reinterpret_cast<uint4*>(a.v_pool + dst);
#pragma unroll 4
        for (int i = lane; i < a.Hkv * D / 8; i += 32) {
            kd[i] = __ldg(ks + i);
            vd[i] = __ldg(vs + i);
        }
        return true;
    };
    // piece number n, once it is published
    auto pieces_done = [&](uint32_t n) {  // the softmax warps are past n pieces
        return until(&sh->epilogues[0], 4 * n) && until(&sh->epilogues[1], 4 * n);
    };
    auto piece_at = [&](uint32_t n, Piece& p) {
        if (!until(&sh->published, n + 1)) return false;
        __threadfence_block();
        p = sh->pieces[n % kPieces];
        return p.t0 < p.t1;
    };

    if (warp >= 8) {
        setmaxnreg_dec<kRegsLow>();
        if (warp == 8) {
            // ------------------------------------------------ MMA issuer
            {
                constexpr uint32_t idesc_s = idesc_bf16_f32(kTileRows, kKeys);
                constexpr uint32_t idesc_o = idesc_bf16_f32(kTileRows, D) | (1u << 16);  // B = V: keys by rows
                const uint32_t q_at = smem_u32(sQ) >> 4, ring_at = smem_u32(ring) >> 4;
                struct Cursor {
                    uint32_t st, ph;  // ring stage and parity of the next K (V) tile
                } kc = {0, 0}, vc = {NK, 0};
                uint32_t fixes = 0;       // per stage: parity of the next fix
                uint32_t q_ph = 0, p_ph = 0, ones = 0;  // parities: bit by Q slot, by warpgroup
                bool ok = true;
                auto wait = [&](uint64_t* bar, uint32_t par) {
                    const bool good = mbar_wait_bounded(bar, par & 1, abort_flag, kWaitNs);
                    if (!good) give_up();
                    ok = __all_sync(0xffffffffu, good) && ok;  // (a later wait may find its phase done)
                    return ok;
                };
                auto wait_q = [&](int s) {
                    const bool good = wait(&sh->q_full[s], q_ph >> s);
                    q_ph ^= 1u << s;
                    return good;
                };
                auto wait_p = [&](int w, int half) {
                    const bool good = wait(&sh->p_full[w][half], p_ph >> w);
                    tc_fence_after();
                    return good;
                };
                // the next K (V) tile is there, and fixed: its stage
                auto take = [&](Cursor& c, bool is_v, bool fixed, uint32_t& stage) {
                    stage = c.st;
                    if (!wait(&sh->full[c.st], c.ph)) return false;
                    if (fixed) {
                        if (!wait(&sh->fix[c.st], fixes >> c.st)) return false;
                        fixes ^= 1u << c.st;
                    }
                    if (++c.st == (is_v ? NST : NK)) {
                        c.st = is_v ? NK : 0;
                        c.ph ^= 1;
                    }
                    tc_fence_after();
                    return true;
                };
                auto free_stage = [&](uint32_t stage) { commit_to(&sh->empty[stage]); };
                // K: 8-row groups, 64-d halves; V, whose dimensions are contiguous,
                // has the halves' distance as its leading offset and steps 16 keys
                auto s_product = [&](int w, int qs, uint32_t stage, bool grouped) {
                    const uint32_t k = ring_at + stage * (Shape::kTile >> 4) + (1u << 16);
                    const uint32_t q = q_at + (uint32_t)qs * (Shape::kTile >> 4) + (1u << 16);
                    const uint32_t half = (grouped ? 1024u : (uint32_t)kHalfBytes) >> 4;
                    const uint32_t hi = kDescHi | (grouped ? 1024u * NH : 1024u) >> 4;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_ss(tmem + w * kKeys, q + (((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4),
                               k + (kk >> 2) * half + (kk & 3) * 2, hi, idesc_s, kk != 0);
                    commit_to(&sh->s_full[w]);
                };
                // O += P.V in two halves of 64 keys, each as soon as its weights are there
                auto pv_product = [&](int w, uint32_t stage, bool grouped, bool first) {
                    const uint32_t half = (grouped ? 1024u : (uint32_t)kHalfBytes) >> 4;
                    const uint32_t v = ring_at + stage * (Shape::kTile >> 4) + (half << 16);
                    const uint32_t hi = kDescHi | (grouped ? 1024u * NH : 1024u) >> 4;
                    const uint32_t step = (grouped ? 2048u * NH : 2048u) >> 4;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (!wait_p(w, h)) return false;
#pragma unroll
                        for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
                            mma_ts(tmem + kTmemO + w * D, tmem + w * kKeys + kk * 8, v + kk * step, hi, idesc_o,
                                   !(first && kk == 0));
                        if (h == 0) commit_to(&sh->pv_half[w]);
                    }
                    p_ph ^= 1u << w;
                    return true;
                };
                Piece p;
                for (uint32_t n = 0; ok && __all_sync(0xffffffffu, until(&sh->checked, n + 1) && piece_at(n, p)); ++n) {
                    const int nt = p.t1 - p.t0;
                    const int kvk = p.kvt - p.t0;  // cached tiles ahead
                    auto grouped = [&](int k) { return a.grouped && k < kvk; };
                    // which tiles the fixing warp touches first
                    const int k_fix = p.merged ? kvk - 1 : -1, v_fix = p.kv % kKeys ? kvk - 1 : -1;
                    const int holed = *(volatile int*)&sh->holed[n % kPieces] ? kvk : nt;
                    const int new_fix = min(holed, kvk + (p.i0 + 1) / kKeys);
                    auto k_fixed = [&](int k) { return k == k_fix || k >= holed; };
                    auto v_fixed = [&](int k) { return k == v_fix || k >= new_fix; };
                    uint32_t ks, vs;
                    // S(k + ...) overwrites P(k), which the product issued before it
                    // reads: the tensor core takes them in this order
                    if (p.mode == kTwo) {
                        if (!wait_q(0) || !wait_q(1) || !take(kc, false, k_fixed(0), ks)) break;
                        s_product(0, 0, ks, grouped(0));
                        s_product(1, 1, ks, grouped(0));
                        free_stage(ks);
                        if (!wait(&sh->o_free[0], n + 1) || !wait(&sh->o_free[1], n + 1)) break;
#pragma unroll 1
                        for (int k = 0; k < nt; ++k) {
                            const bool more = k + 1 < nt;
                            if (!take(vc, true, v_fixed(k), vs) || (more && !take(kc, false, k_fixed(k + 1), ks))) break;
#pragma unroll 1
                            for (int w = 0; w < 2; ++w) {
                                if (!pv_product(w, vs, grouped(k), k == 0)) break;
                                if (more) s_product(w, w, ks, grouped(k + 1));
                            }
                            free_stage(vs);
                            if (more) free_stage(ks);
                        }
                        for (int w = 0; w < 2; ++w) {
                            commit_to(&sh->pv_done[w]);
                            commit_to(&sh->q_empty[w]);
                        }
                    } else {
                        const int qs = ones++ & 1;
                        auto s_next = [&](int k) {
                            if (k >= nt) return true;
                            if (!take(kc, false, k_fixed(k), ks)) return false;
                            s_product(k & 1, qs, ks, grouped(k));
                            free_stage(ks);
                            return true;
                        };
                        if (!wait_q(qs) || !s_next(0) || !s_next(1)) break;
                        if (!wait(&sh->o_free[0], n + 1) || !wait(&sh->o_free[1], n + 1)) break;
#pragma unroll 1
                        for (int k = 0; k < nt; ++k) {
                            if (!take(vc, true, v_fixed(k), vs) || !pv_product(k & 1, vs, grouped(k), k < 2)) break;
                            free_stage(vs);
                            if (k + 2 >= nt) commit_to(&sh->pv_done[k & 1]);
                            if (!s_next(k + 2)) break;
                        }
                    }
                }
                commit_to(&sh->drain);
                mbar_wait_bounded(&sh->drain, 0, &sh->never, kWaitNs);
            }
        } else if (warp <= 10) {
            // ------------------------------------------------ TMA producers
            // Warp 9 walks the CTA's range (order: request, KV head, item),
            // publishes its pieces to the other roles and loads the K tiles; warp
            // 10 loads Q and the V tiles.
            const bool is_v = warp == 10;
            const uint64_t pol = policy_evict_normal(), pol_first = policy_evict_first();
            uint32_t st = is_v ? NK : 0, ph = 0, armed = 0, armed_ph = 0;  // the next tile's stage and parity; stages loaded into
            uint32_t tiles = 0, n = 0, q_use[2] = {0, 0}, ones = 0;
            const int nb = kKeys / a.box;  // boxes of a cached tile (of each 64-d half, when not grouped)
            const int x_row = (lane < nb ? lane : 0) * a.box;
            const int tile_pages = kKeys / a.P, tile_rest = kKeys % a.P;
            const int none = (int)((long long)a.num_pages * a.P / kGroupRows);  // the group past the last: reads as zeros
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t par) {
                if (lane == 0 && !mbar_wait_bounded(bar, par & 1, abort_flag, kWaitNs)) {
                    give_up();
                    ok = false;
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                return ok;
            };
            auto publish = [&](const Piece& p) {
                // the roles that might lag are done with the record's old piece
                if (n >= kPieces) {
                    ok = until(&sh->fixed, n - kPieces + 1) && pieces_done(n - kPieces + 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) return;
                }
                if (lane == 0) {
                    sh->pieces[n % kPieces] = p;
                    __threadfence_block();
                    *(volatile uint32_t*)&sh->published = n + 1;
                }
                __syncwarp();
            };
            int b = bad ? a.B : sh->b, g = sh->g, q = sh->q;
            long long rel = sh->rel;  // the item's start less my0
            const long long len = sh->len;
            Request r = sh->first;
            // the next piece of the walk; one without tiles at its end
            auto walk = [&](Piece& p) {
                p.t0 = p.t1 = 0;
                while (b < a.B && rel < len) {
                    const Item it = item_of(a, r, q);
                    const long long start = rel;
                    cut_tiles(it, start, len, p.t0, p.t1);
                    p.b = b;
                    p.g = g;
                    p.start = r.start;
                    p.kv = r.kv;
                    p.kvt = r.kvt;
                    p.i0 = it.i0;
                    p.i1 = it.i1;
                    p.mode = it.two ? kTwo : it.i1 - it.i0 <= a.tps ? kQuad : kOne;
                    p.slot = p.t0 > 0 ? 0 : p.t1 < it.nt ? 1 : -1;
                    p.merged = r.merged;
                    p.items = r.items;
                    // the next item
                    rel += it.cost;
                    if (++q >= r.items) {
                        q = 0;
                        if (++g >= a.Hkv) {
                            g = 0;
                            do {
                                if (++b >= a.B) break;
                                r = request_of(a, a.q_start[b], a.q_start[b + 1], a.kv_len[b]);
                            } while (r.items == 0);
                        }
                    }
                    if (p.t0 < p.t1) {
                        if (p.slot == 1 && lane == 0) {
                            // CTAs that hold a part: this one to the owner of the item's last tile
                            const int G = cut_ctas(a, sh->total, gridDim.x);
                            const int last =
                                cut_owner(sh->total, G, sh->my0 + start + (long long)(it.nt - 1) * it.w);
                            ChunkCut c = {last - (int)blockIdx.x + 1, p.g, it.i0, it.i1, p.start, {0, 0, 0}};
                            a.cuts[blockIdx.x] = c;
                        }
                        return;
                    }
                    p.t0 = p.t1 = 0;
                }
            };
            for (; ok; ++n) {
                Piece p;
                if (!is_v) {
                    walk(p);
                    publish(p);
                    if (!ok || p.t0 >= p.t1) break;
                } else {
                    if (!__all_sync(0xffffffffu, piece_at(n, p))) break;
                    const bool two = p.mode == kTwo, quad = p.mode == kQuad;
                    const int q0 = two ? 0 : ones++ & 1, q1 = two ? 1 : q0;
                    for (int s = q0; s <= q1; ++s) {
                        if (!wait(&sh->q_empty[s], q_use[s] + 1)) break;
                        ++q_use[s];
                        // of 32 rows four copies, else one; each in 64-d halves
                        const int copies = quad ? 4 : 1;
                        if (lane == 0)
                            mbar_arrive_expect_tx(&sh->q_full[s],
                                                  (uint32_t)((quad ? 4 * a.tps : a.tpq) * a.grp * 128 * NH));
                        __syncwarp();
                        if (lane < copies * NH) {
                            const int h = lane / copies, c = lane - h * copies;
                            tma_load_4d(sQ + s * Shape::kTile + h * kHalfBytes + c * 32 * 128, quad ? &tm_qs : &tm_q,
                                        &sh->q_full[s], 64 * h, p.g * a.grp, p.start + p.i0 + (s - q0) * a.tpq, 0, pol);
                        }
                    }
                    if (!ok) break;
                }
                // lane x holds the page of box x, rows from x * box on, of a
                // grouped tile (keys past the cached ones have none; such a page,
                // like a bad one, reads as zeros); the next tile's is fetched while
                // one is loaded
                const int32_t* table = a.page_table + (size_t)p.b * a.max_pages;
                auto checked = [&](int page) {
                    if (page >= 0 && page < a.num_pages) return page;
                    raise_flag(a.err_flag, ISD_FLAG_PAGE_OOB);
                    return -1;
                };
                int key = p.t0 * kKeys + x_row, at = key / a.P, in = key - at * a.P, page = 0;
                if (a.grouped && key < p.kv) page = __ldg(table + at);
                // keys that only this item reads need not stay in L2
                const uint64_t pol_kv = p.items == 1 ? pol_first : pol;
                const CUtensorMap* map = is_v ? &tm_v : &tm_k;
#pragma unroll 1
                for (int t = p.t0; t < p.t1; ++t) {
                    int group = none;
                    if (key < p.kv && a.grouped) {
                        const int id = checked(page);
                        if (id >= 0) group = (int)(((long long)id * a.P + in) / kGroupRows);
                    }
                    if (a.grouped && t + 1 < p.t1) {
                        key += kKeys;
                        at += tile_pages;
                        in += tile_rest;
                        if (in >= a.P) {
                            in -= a.P;
                            ++at;
                        }
                        if (key < p.kv) page = __ldg(table + at);
                    }
                    if (!wait(&sh->empty[st], ph ^ 1)) break;
                    unsigned char* dst = ring + st * Shape::kTile;
                    uint64_t* bar = &sh->full[st];
                    ++tiles;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar, Shape::kTile);
                        *(volatile uint32_t*)&sh->issued[is_v] = tiles;
                    }
                    armed |= 1u << st;
                    armed_ph = (armed_ph & ~(1u << st)) | ph << st;
                    if (++st == (is_v ? NST : NK)) {
                        st = is_v ? NK : 0;
                        ph ^= 1;
                    }
                    __syncwarp();
                    if (t >= p.kvt) {
                        if (lane < NH)
                            tma_load_4d(dst + lane * kHalfBytes, is_v ? &tm_vn : &tm_kn, bar, 64 * lane, p.g,
                                        p.start + (t - p.kvt) * kKeys, 0, pol);
                    } else if (a.grouped) {
                        if (lane < nb)
                            tma_load_4d(dst + x_row * (128 * NH), map, bar, 0, 0, p.g * NH, group, pol_kv);
                    } else {
                        for (int x = lane; x < nb * NH; x += 32) {
                            const int h = x / nb, row = (x - h * nb) * a.box, k = t * kKeys + row;
                            tma_load_4d(dst + h * kHalfBytes + row * 128, map, bar, 64 * h, p.g, k % a.P,
                                        k < p.kv ? checked(__ldg(table + k / a.P)) : -1, pol_kv);
                        }
                    }
                }
            }
            // drain: every copy has landed before the CTA may exit
            if (lane == 0) {
                for (int s = 0; s < NST; ++s)
                    if (armed >> s & 1) mbar_wait_bounded(&sh->full[s], armed_ph >> s & 1, &sh->never, kWaitNs);
                for (int s = 0; s < 2; ++s)
                    if (q_use[s]) mbar_wait_bounded(&sh->q_full[s], (q_use[s] - 1) & 1, &sh->never, kWaitNs);
            }
        } else {
            // ------------------------------------------------ tiles that need a touch
            // before a product may read them: rows that hold no key of the item
            // are zeroed in V (0 * NaN would spoil the sum), the new tokens of a
            // merged tile are put into their rows, and infinities and NaN in V
            // rows that only some of the item's rows see are taken out and noted
            // for the epilogue.  What a page outside the pool would hold counts as
            // zeros, new or cached: where a request has new tokens on one, their
            // rows are zeroed in all its tiles of new tokens.
            uint32_t tiles = 0, n = 0;  // key tiles of the pieces before; pieces
            bool ok = true, more_new = true;
            auto all_ok = [&](bool good) {
                ok = __all_sync(0xffffffffu, good);
                return ok;
            };
            // The tile (K: v = 0, V: v = 1) number `tile` of this CTA has landed.
            // This warp skips most, so it first waits until the producer is at
            // this one: the barrier's phase is then the tile's, and stays it until
            // the fix.
            auto landed = [&](int v, uint32_t tile) {
                // (after its first piece it spends the time appending)
                while (n && more_new && !__any_sync(0xffffffffu, peek(&sh->issued[v]) > tile)) more_new = append();
                if (!all_ok(until(&sh->issued[v], tile + 1))) return false;
                const uint32_t s = v ? NK + tile % NV : tile % NK, round = v ? tile / NV : tile / NK;
                const bool good = mbar_wait_bounded(&sh->full[s], round & 1, abort_flag, kWaitNs);
                if (!good) give_up();
                return all_ok(good);
            };
            auto done = [&](uint32_t s) {
                proxy_fence();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->fix[s]);
            };
            constexpr int kChunks = D / 8;           // 16-byte chunks of a row
            constexpr int kRowsStep = 32 / kChunks;  // rows the warp covers at once
            const int ch = lane % kChunks, r_in = lane / kChunks;
            auto cell = [&](uint32_t s, int row, bool grouped) {
                const int at = grouped ? (row >> 3) * (1024 * NH) + (ch >> 3) * 1024 + (row & 7) * 128
                                       : (ch >> 3) * kHalfBytes + row * 128;
                return reinterpret_cast<uint4*>(ring + s * Shape::kTile + at + (((ch & 7) ^ (row & 7)) << 4));
            };
            // notes what is not finite in this lane's chunk of token `tok` and returns the chunk without it
            auto note = [&](uint4 w, int tok) {
                uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t half = (x[i >> 1] >> (16 * (i & 1))) & 0xffffu;
                    if ((half & 0x7f80u) != 0x7f80u) continue;
                    const int kind = (half & 0x7fu) ? 2 : (half >> 15);
                    atomicMin(&sh->bad_from[kind][ch * 8 + i], tok);
                    x[i >> 1] &= ~(0xffffu << (16 * (i & 1)));
                }
                return make_uint4(x[0], x[1], x[2], x[3]);
            };
            // makes `bad_from` this piece's, once every earlier piece has read its own
            auto claim = [&]() {
                if (sh->bad_piece == (int)n) return true;
                if (!all_ok(pieces_done(n))) return false;
                for (int i = lane; i < 3 * D; i += 32) (&sh->bad_from[0][0])[i] = 0x7fffffff;
                __syncwarp();
                if (lane == 0) *(volatile int*)&sh->bad_piece = (int)n;
                __syncwarp();
                return true;
            };
            auto outside = [&](int page) { return page < 0 || page >= a.num_pages; };
            int new_b = -1, new_n = 0;  // whether some of request new_b's first new_n new
            bool holes = false;         // tokens lie on a page outside the pool
            Piece p;
            while (all_ok(piece_at(n, p))) {
                const int32_t* table = a.page_table + (size_t)p.b * a.max_pages;
                if (p.t1 > p.kvt && (p.b != new_b || p.i1 > new_n)) {
                    if (p.b != new_b) new_n = holes = 0;
                    const int to = (p.kv + p.i1 - 1) / a.P;
#pragma unroll 8
                    for (int c = (p.kv + new_n) / a.P + lane; c <= to; c += 32) holes |= outside(__ldg(table + c));
                    holes = __any_sync(0xffffffffu, holes);
                    new_b = p.b;
                    new_n = p.i1;
                }
                const bool holed = p.t1 > p.kvt && holes;
                if (lane == 0) {
                    *(volatile int*)&sh->holed[n % kPieces] = holed;
                    __threadfence_block();
                    *(volatile uint32_t*)&sh->checked = n + 1;
                }
                // the cached tile with free rows, and the new tiles that some row does not see whole
                if (p.kv % kKeys && p.t0 < p.kvt && p.t1 >= p.kvt) {
                    const uint32_t tile = tiles + (p.kvt - 1 - p.t0);
                    const uint32_t ks = tile % NK, vs = NK + tile % NV;
                    const int m = p.kv % kKeys;  // cached keys of the tile
                    // the item's new tokens (a row of an item sees none past its last)
                    const int fresh = p.merged ? p.i1 : 0;
                    uint32_t zeros = 0;  // bit i: token i lies on a page outside the pool
                    auto new_chunk = [&](const __nv_bfloat16* src, int i) {
                        return __ldg(reinterpret_cast<const uint4*>(src + ((size_t)(p.start + i) * a.Hkv + p.g) * D) + ch);
                    };
                    uint4 k_next = make_uint4(0, 0, 0, 0), v_next = k_next;  // fetched while the tile is on its way
                    if (fresh) {
                        int id = 0;
                        if (lane < fresh) id = __ldg(table + (p.kv + lane) / a.P);
                        if (r_in < fresh) {
                            k_next = new_chunk(a.k_new, r_in);
                            v_next = new_chunk(a.v_new, r_in);
                        }
                        if (!landed(0, tile)) break;
                        zeros = __ballot_sync(0xffffffffu, outside(id));
                        for (int i = r_in; i < fresh; i += kRowsStep) {
                            *cell(ks, m + i, a.grouped) = zeros >> i & 1 ? make_uint4(0, 0, 0, 0) : k_next;
                            if (i + kRowsStep < fresh) k_next = new_chunk(a.k_new, i + kRowsStep);
                        }
                        done(ks);
                    }
                    if (!landed(1, tile)) break;
                    for (int i0 = 0; i0 < fresh; i0 += kRowsStep) {
                        const int i = i0 + r_in;
                        uint4 w = v_next;
                        if (i < fresh && (zeros >> i & 1)) w = make_uint4(0, 0, 0, 0);
                        if (i + kRowsStep < fresh) v_next = new_chunk(a.v_new, i + kRowsStep);
                        else v_next = make_uint4(0, 0, 0, 0);
                        const bool odd = odd_bits(w) & kOddBits;
                        if (__any_sync(0xffffffffu, odd)) {
                            if (!claim()) break;
                            if (odd) w = note(w, i);
                        }
                        if (i < fresh) *cell(vs, m + i, a.grouped) = w;
                    }
                    if (!ok) break;
                    for (int row = m + fresh + r_in; row < kKeys; row += kRowsStep)
                        *cell(vs, row, a.grouped) = make_uint4(0, 0, 0, 0);
                    done(vs);
                }
                const int first = max(p.t0, p.kvt + (holed ? 0 : p.i0 / kKeys));
                for (int t = first; ok && t < p.t1; ++t) {
                    const int base = (t - p.kvt) * kKeys;
                    const bool whole = base + kKeys <= p.i0 + 1;  // every row sees all of it
                    if (whole && !holed) continue;
                    const uint32_t tile = tiles + (t - p.t0), vs = NK + tile % NV;
                    const int rows = min(kKeys, p.i1 - base);
                    auto zero_holes = [&](uint32_t s) {
                        for (int row = r_in; row < rows; row += kRowsStep)
                            if (outside(__ldg(table + (p.kv + base + row) / a.P))) *cell(s, row, false) = make_uint4(0, 0, 0, 0);
                        __syncwarp();
                    };
                    if (__builtin_expect(holed, 0)) {
                        if (!landed(0, tile)) break;
                        zero_holes(tile % NK);
                        done(tile % NK);
                        if (!landed(1, tile)) break;
                        zero_holes(vs);
                        if (whole) {
                            done(vs);
                            continue;
                        }
                    }
                    if (!landed(1, tile)) break;
                    // a first pass over the rows looks for anything odd, eight loads at
                    // once; what it finds (hardly ever) is taken out one by one
                    uint32_t odd_any = 0;
                    const int r0 = max(0, p.i0 + 1 - base);
#pragma unroll 8
                    for (int row = r0 + r_in; row < rows; row += kRowsStep) odd_any |= odd_bits(*cell(vs, row, false));
                    if (__builtin_expect(__any_sync(0xffffffffu, odd_any & kOddBits), 0)) {
                        if (!claim()) break;
                        for (int row = r0 + r_in; row < rows; row += kRowsStep) {
                            const uint4 w = *cell(vs, row, false);
                            if (odd_bits(w) & kOddBits) *cell(vs, row, false) = note(w, base + row);
                        }
                    }
                    if (!ok) break;
                    for (int row = rows + r_in; row < kKeys; row += kRowsStep)
                        *cell(vs, row, false) = make_uint4(0, 0, 0, 0);
                    done(vs);
                }
                if (!ok) break;
                tiles += p.t1 - p.t0;
                ++n;
                if (lane == 0) *(volatile uint32_t*)&sh->fixed = n;
            }
            if (lane == 0) *(volatile uint32_t*)&sh->checked = n + 1;  // (the end of the pieces)
            while (more_new) more_new = append();
        }
    } else {
        setmaxnreg_inc<kRegsHigh>();
        // While the first tiles are on their way: a new token per warp.
        if (!bad) append();
        // ---------------------------------------------------- softmax and epilogue
        const int wg = warp >> 2, wq = warp & 3;  // warpgroup; its warp, a quarter of the TMEM lanes
        const uint32_t tm_lane = tmem + ((uint32_t)(wq * 32) << 16);
        const uint32_t tm_s = tm_lane + wg * kKeys, tm_o = tm_lane + kTmemO;
        uint32_t s_use = 0, o_use = 0, ones = 0, met = 0;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t par) {
            const bool good = mbar_wait_bounded(bar, par & 1, abort_flag, kWaitNs);
            if (!good) give_up();
            ok = __all_sync(0xffffffffu, good);
            return ok;
        };
        // barrier of the eight softmax warps (a bounded one, like every wait)
        auto soft_sync = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->meet);
            return wait(&sh->meet, met++);
        };
        Piece p;
        for (uint32_t n = 0; ok && __all_sync(0xffffffffu, piece_at(n, p)); ++n) {
            const bool quad = p.mode == kQuad;
            const int rr = quad ? lane : wq * 32 + lane;  // row in its tile
            const int tok = (p.mode == kTwo ? wg * a.tpq : 0) + rr / a.grp;
            const int i = p.i0 + tok;  // this row's token
            const bool live = rr < (quad ? a.tps : a.tpq) * a.grp && i < p.i1;
            const int step = p.mode == kTwo ? 1 : 2, t_first = p.t0 + (p.mode == kTwo ? 0 : wg);
            float m_ref = -INFINITY, l = 0.f;
            // the row's maximum is top: the reference, l, and O if it holds products,
            // follow.  (The maximum's own weight is then 1 but for the reference's
            // rounding, half a step of its 32 bits: 1 +- 1.7e-4 at references of 4096
            // to 8192, which is 1 in bf16.)
            auto move_ref = [&](float top, bool has_o) {
                const float m_new = fmaxf(m_ref, top);
                const float f = m_new > m_ref ? ex2(m_ref - m_new) : 1.f;
                if (has_o) {
#pragma unroll 1
                    for (int j = 0; j < D; j += 16) {
                        uint32_t o[16];
                        tmem_ld16(tm_o + wg * D + j, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st16(tm_o + wg * D + j, o);
                    }
                    tmem_st_wait();
                }
                l *= f;
                m_ref = m_new;
            };
            auto hide = [&](float (&s)[32], bool some, int seen) {  // scores from `seen` on
                if (some) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j >= seen) s[j] = -INFINITY;
                }
            };
            auto top_of = [&](const float (&s)[32]) {
                float x = fmaxf(s[0], s[1]), y = fmaxf(s[2], s[3]);
#pragma unroll
                for (int j = 4; j < 32; j += 4) {
                    x = fmaxf(x, fmaxf(s[j], s[j + 1]));
                    y = fmaxf(y, fmaxf(s[j + 2], s[j + 3]));
                }
                return fmaxf(x, y);
            };
            // weights of 32 scores: summed in 32 bits, and rounded to bf16 for the
            // product with V, whose operands have one type (V's).  A weight is off by
            // half a bf16 step, 2^-8 of itself: against 64 bits results are off by
            // 0.0020 to 0.0023 (norm), of which their own rounding is 0.0016; keeping
            // the weights' low halves too would double the product.  (The
            // special-function unit, 16 exponentials a clock and SM, is what two warps
            // on a sub-partition wait for here: 522 cycles for 32 scores each, one alone
            // 302.  Taking a part of them by a polynomial on the FMA pipes, which costs
            // 22 cycles a pair against 16, measured 475 to 500 at best, and no gain for
            // the whole kernel.)
            auto weights = [&](const float (&s)[32], float mu, unsigned long long& sum, uint32_t* w) {
                const unsigned long long sc = pair(a.scale_log2, a.scale_log2), neg = pair(-mu, -mu);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float x, y;
                    unpair(fma2(pair(s[2 * j], s[2 * j + 1]), sc, neg), x, y);
                    x = ex2(x);
                    y = ex2(y);
                    sum = add2(sum, pair(x, y));
                    w[j] = pack_bf16(x, y);
                }
            };
            auto mu_of = [&]() { return m_ref == -INFINITY ? 0.f : m_ref; };
            auto sum_of = [](unsigned long long acc) {
                float x, y;
                unpair(acc, x, y);
                return x + y;
            };
            auto hand_over = [&](int half) {
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->p_full[wg][half]);
            };
            // The next tile's scores are here (and so the warpgroup's product before
            // them is done).  Whether some of its keys are hidden from some row, and
            // how many this row sees:
            auto arrived = [&]() {
                const bool good = wait(&sh->s_full[wg], s_use++);
                tc_fence_after();
                return good;
            };
            auto partly = [&](int t) {
                return t < p.kvt ? (t + 1) * kKeys > p.kv : (t + 1 - p.kvt) * kKeys > p.i0 + 1;
            };
            auto seen_of = [&](int t) {
                if (t >= p.kvt) return i + 1 - (t - p.kvt) * kKeys;
                return p.kv - t * kKeys + (p.merged && t == p.kvt - 1 ? i + 1 : 0);
            };
            // Weights are taken by the reference as it is.  Only when there is none yet,
            // or a row's sum of them passes 2^10 (then one may be large) or is NaN, is its maximum
            // looked up, the reference moved, and the weights are done over: S is
            // still there.
            if (quad) {
                for (int t = t_first; t < p.t1; t += step) {
                    if (!arrived()) break;
                    // a quarter of the keys: the row's other quarters are other warps'
                    const bool has_o = t != t_first;
                    float s[32];
                    tmem_ld32(tm_s + wq * 32, s);
                    tmem_arrived(s);
                    hide(s, partly(t), seen_of(t) - wq * 32);
                    // a row's first scores set its reference (a quarter may have seen none so far)
                    if (__any_sync(0xffffffffu, live && m_ref == -INFINITY)) move_ref(top_of(s) * a.scale_log2, has_o);
                    uint32_t w[16];
                    float sum;
#pragma unroll 1
                    for (int round = 0;; ++round) {
                        unsigned long long acc = 0;
                        weights(s, mu_of(), acc, w);
                        sum = sum_of(acc);
                        if (__builtin_expect(round || !__any_sync(0xffffffffu, live && sum > 1024.f), 1)) break;
                        move_ref(top_of(s) * a.scale_log2, has_o);
                    }
                    l += sum;
                    const uint32_t zero[16] = {};
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (c != wq) tmem_st16(tm_s + c * 16, zero);
                    tmem_st16(tm_s + wq * 16, w);
                    hand_over(0);
                    hand_over(1);
                }
            } else {
                for (int t = t_first; t < p.t1; t += step) {
                    if (!arrived()) break;
                    const bool has_o = t != t_first, some = partly(t);
                    float s0[32];
                    int h_done = 0;
                    // moves the reference if a maximum of these scores passes it by `over`
                    auto look = [&](int from, int to, float over, bool has_o) {
                        float top = -INFINITY;
#pragma unroll 1
                        for (int c = from; c < to; c += 32) {
                            tmem_ld32(tm_s + c, s0);
                            tmem_arrived(s0);
                            hide(s0, some, seen_of(t) - c);
                            top = fmaxf(top, top_of(s0));
                        }
                        top *= a.scale_log2;
                        // (rows that are no one's have whatever is in Q: they decide nothing)
                        if (__any_sync(0xffffffffu, live && top > m_ref + over)) move_ref(top, has_o);
                    };
                    if (__builtin_expect(!has_o || some, 0)) look(0, kKeys, has_o ? 8.f : 0.f, has_o);
                    // half by half; P takes the place of scores already read
                    if (__builtin_expect(!some, 1)) {
                        tmem_ld32(tm_s, s0);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int c = h * 64;
                            const float mu = mu_of();
                            unsigned long long acc = 0;
                            uint32_t w[32];
                            float s1[32];
                            tmem_arrived(s0);
                            tmem_ld32(tm_s + c + 32, s1);
                            weights(s0, mu, acc, w);
                            tmem_arrived(s1);
                            if (h == 0) tmem_ld32(tm_s + 64, s0);
                            weights(s1, mu, acc, w + 16);
                            const float sum = sum_of(acc);
                            if (__builtin_expect(__any_sync(0xffffffffu, live && (!(sum <= 1024.f) || m_ref == -INFINITY)), 0)) {
                                if (h == 0) tmem_arrived(s0);
                                break;
                            }
                            l += sum;
                            tmem_st32(tm_s + c / 2, w);
                            hand_over(h);
                            h_done = h + 1;
                        }
                    }
#pragma unroll 1
                    for (int h = h_done; h < 2; ++h) {
                        const int c = h * 64;
                        if (!some) {
                            // O has to stand still: the first half's product may be under way
                            if (h == 1 && !wait(&sh->pv_half[wg], s_use - 1)) break;
                            tc_fence_after();
                            look(c, c + 64, 0.f, has_o || h == 1);
                        }
                        unsigned long long acc = 0;
#pragma unroll 1
                        for (int j = 0; j < 2; ++j) {
                            uint32_t w[16];
                            tmem_ld32(tm_s + c + 32 * j, s0);
                            tmem_arrived(s0);
                            hide(s0, some, seen_of(t) - c - 32 * j);
                            weights(s0, mu_of(), acc, w);
                            tmem_st16(tm_s + c / 2 + 16 * j, w);
                        }
                        l += sum_of(acc);
                        hand_over(h);
                    }
                    if (!ok) break;
                }
            }
            if (!ok) break;
            // ---- this piece's rows
            if (t_first < p.t1 && !wait(&sh->pv_done[wg], o_use++)) break;
            tc_fence_after();
            if (p.mode != kTwo) {
                // a warpgroup may have no tile of the piece: the other one's
                // products are done too
                tc_fence_before();
                if (!soft_sync()) break;
                tc_fence_after();
            }
            const bool odd = *(volatile int*)&sh->bad_piece == (int)n;
            auto spoil = [&](float v, int d) {  // what the fixing warp took out, for the rows that see it
                if (sh->bad_from[0][d] <= i) v += INFINITY;
                if (sh->bad_from[1][d] <= i) v -= INFINITY;
                if (sh->bad_from[2][d] <= i) v = NAN;
                return v;
            };
            __nv_bfloat16* orow = a.out + ((size_t)(p.start + i) * a.Hq + p.g * a.grp + rr % a.grp) * D;
            float* part = a.part + ((size_t)blockIdx.x * 2 + max(p.slot, 0)) * (size_t)a.part_rows * (D + 2);
            const int prow = (p.mode == kTwo ? wg * kTileRows : 0) + rr;
            // 8 dimensions of a finished row, or of its part
            auto store8 = [&](float (&v)[8], int d, float inv) {
                if (__builtin_expect(odd, 0)) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = spoil(v[e], d + e);
                }
                if (!live) return;
                if (p.slot >= 0) {
                    float4* po = reinterpret_cast<float4*>(part + 2 * a.part_rows) + (size_t)(d / 4) * a.part_rows + prow;
                    po[0] = make_float4(v[0], v[1], v[2], v[3]);
                    po[a.part_rows] = make_float4(v[4], v[5], v[6], v[7]);
                } else {
                    *reinterpret_cast<uint4*>(orow + d) =
                        make_uint4(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv),
                                   pack_bf16(v[4] * inv, v[5] * inv), pack_bf16(v[6] * inv, v[7] * inv));
                }
            };
            if (p.mode == kTwo) {
                if (p.slot >= 0 && live) {
                    part[prow] = m_ref;
                    part[a.part_rows + prow] = l;
                }
                const float inv = 1.f / l;
                const bool wide = ((uintptr_t)a.out & 31) == 0;
#pragma unroll 1
                for (int d = 0; d < D; d += 16) {
                    uint32_t u[16];
                    tmem_ld16(tm_o + wg * D + d, u);
                    tmem_ld_wait();
                    float o[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __uint_as_float(u[e]);
                    if (__builtin_expect(odd, 0)) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = spoil(o[e], d + e);
                    }
                    if (!live) continue;
                    if (p.slot >= 0) {
                        float4* po = reinterpret_cast<float4*>(part + 2 * a.part_rows) + (size_t)(d / 4) * a.part_rows + prow;
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            po[(size_t)(e / 4) * a.part_rows] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    } else {
                        uint32_t h[8];
#pragma unroll
                        for (int x = 0; x < 8; ++x) h[x] = pack_bf16(o[2 * x] * inv, o[2 * x + 1] * inv);
                        store32(orow + d, h, wide);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_n(&sh->o_free[wg], 2);
            } else {
                // both warpgroups hold a part of the rows (and, of 32 rows, every
                // warp): they meet in the item's Q tile, whose products are done
                const int qs = ones++ & 1;
                float* meet = reinterpret_cast<float*>(sQ + qs * Shape::kTile);
                // maxima and sums: [8][32] each, by warp, of its 32 rows
                meet[warp * 32 + lane] = m_ref;
                meet[256 + warp * 32 + lane] = l;
                if (!soft_sync()) break;
                const int w0 = quad ? 0 : wq, ws = quad ? 1 : 4;  // the warps that share this thread's row
                float top = -INFINITY, sum = 0.f;
#pragma unroll 1
                for (int w = w0; w < 8; w += ws) top = fmaxf(top, meet[w * 32 + lane]);
                const float mu = top == -INFINITY ? 0.f : top;
#pragma unroll 1
                for (int w = w0; w < 8; w += ws) sum += meet[256 + w * 32 + lane] * ex2(meet[w * 32 + lane] - mu);
                const float inv = 1.f / sum;
                const float f0 = ex2(meet[wq * 32 + lane] - mu), f1 = ex2(meet[(4 + wq) * 32 + lane] - mu);
                if (p.slot >= 0 && live && wg == 0 && (!quad || wq == 0)) {
                    part[prow] = top;
                    part[a.part_rows + prow] = sum;
                }
                // 8 dimensions of both warpgroups' O; a part of no weight counts for
                // nothing, whatever it holds
                auto both8 = [&](int d, float (&v)[8]) {
                    uint32_t x[8], y[8];
                    tmem_ld8(tm_o + d, x);
                    tmem_ld8(tm_o + D + d, y);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = (f0 > 0.f ? __uint_as_float(x[e]) * f0 : 0.f) +
                               (f1 > 0.f ? __uint_as_float(y[e]) * f1 : 0.f);
                };
                if (!quad) {
#pragma unroll 1
                    for (int d = wg * (D / 2); d < (wg + 1) * (D / 2); d += 8) {
                        float v[8];
                        both8(d, v);
                        store8(v, d, inv);
                    }
                } else {
                    // the four quarters through shared memory, `width` dimensions at
                    // a time: [4][rows][width + 1]
                    float* stage = meet + 512;
                    const int rows = (p.i1 - p.i0) * a.grp;
                    const int width = rows <= 8 ? D : D / 4;
#pragma unroll 1
                    for (int d0 = 0; d0 < D; d0 += width) {
#pragma unroll 1
                        for (int d = wg * (width / 2); d < (wg + 1) * (width / 2); d += 8) {
                            float v[8];
                            both8(d0 + d, v);
                            if (live) {
#pragma unroll
                                for (int e = 0; e < 8; ++e) stage[(wq * rows + lane) * (width + 1) + d + e] = v[e];
                            }
                        }
                        if (!soft_sync()) break;
                        // a row per thread again, 8 dimensions each: warps take slices
                        if (live) {
#pragma unroll 1
                            for (int d = warp * 8; d < width; d += 64) {
                                float v[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const float* x = stage + lane * (width + 1) + d + e;
                                    const int q1 = rows * (width + 1);
                                    v[e] = (x[0] + x[q1]) + (x[2 * q1] + x[3 * q1]);
                                }
                                store8(v, d0 + d, inv);
                            }
                        }
                        if (!soft_sync()) break;
                    }
                }
                tc_fence_before();
                proxy_fence();
                if (!ok || !soft_sync()) break;
                if (threadIdx.x == 0) mbar_arrive(&sh->q_empty[qs]);
                if (lane == 0) {
                    mbar_arrive(&sh->o_free[0]);
                    mbar_arrive(&sh->o_free[1]);
                }
            }
            if (lane == 0) atomicAdd(&sh->epilogues[wg], 1u);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Running maximum, sum and weighted values of a row: another part joins them.
template <int N>
ISD_DEVINL void join_part(float& m, float& l, float (&o)[N], float mk, float lk, const float (&ok)[N]) {
    const float mn = fmaxf(m, mk), mu = mn == -INFINITY ? 0.f : mn;
    const float f0 = ex2(m - mu), f1 = ex2(mk - mu);
    l = l * f0 + lk * f1;
#pragma unroll
    for (int e = 0; e < N; ++e)  // a part of no weight counts for nothing
        o[e] = (f0 > 0.f ? o[e] * f0 : 0.f) + (f1 > 0.f ? ok[e] * f1 : 0.f);
    m = mn;
}

// Joins the parts of cut items, always in the same order: grid (CTAs, 32-row
// groups, slices of the dimensions), a lane per row.  Of few parts a warp joins
// D / 8 dimensions, the loads of two parts in flight.  Of more (a long context)
// `share` warps take the parts in turn, for 16 dimensions, and meet in shared
// memory.  With many rows the blocks hide each other's loads, so the first way
// holds up to kJoinMany parts: 2048 tokens at once took 8 us of the call against
// 12 by the second way, prompts of 3 to 333 tokens with 64-wide heads 5 against
// 12.  With few rows it holds up to kJoinFew: one token behind 1000 took 3.4 us by
// the second way against 5 by the first.
constexpr int kJoinWarps = 8, kJoinDims = 16, kJoinFew = 3, kJoinMany = 16;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) chunk_join_kernel(const __grid_constant__ ChunkArgs a) {
    __shared__ float red[kJoinWarps][kJoinDims + 2][32];
    pdl_wait();  // (and no early trigger: the next call's CTAs among these cost 2 to 6% with many rows)
    const ChunkCut cut = a.cuts[blockIdx.x];
    if (cut.parts < 2) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.y * 32 + lane, rr = row % kTileRows;
    const int i = cut.i0 + row / kTileRows * a.tpq + rr / a.grp;
    const bool live = rr < a.tpq * a.grp && i < cut.i1;
    if (!__any_sync(0xffffffffu, live)) return;  // the same lanes in every warp
    const size_t stride = (size_t)a.part_rows * (D + 2);
    const float* first = a.part + ((size_t)blockIdx.x * 2 + 1) * stride;
    // part k: the first one in slot 1 of its CTA, the others in slot 0 of theirs
    auto part = [&](int k) { return k == 0 ? first : first + (size_t)(2 * k - 1) * stride; };
    auto load = [&](const float* pk, int d, float* to, int count) {
        const float4* po = reinterpret_cast<const float4*>(pk + 2 * a.part_rows) + (size_t)(d / 4) * a.part_rows + row;
#pragma unroll
        for (int e = 0; e < count; e += 4) {
            const float4 v = po[(size_t)(e / 4) * a.part_rows];
            to[e] = v.x;
            to[e + 1] = v.y;
            to[e + 2] = v.z;
            to[e + 3] = v.w;
        }
    };
    __nv_bfloat16* out = a.out + ((size_t)(cut.start + i) * a.Hq + cut.g * a.grp + rr % a.grp) * D;
    if (cut.parts <= (a.part_rows > kTileRows ? kJoinMany : kJoinFew)) {
        if (!live || blockIdx.z) return;
        constexpr int N = D / kJoinWarps, kBatch = 2;
        const int d0 = warp * N;
        float m = -INFINITY, l = 0.f, o[N] = {};
        for (int k0 = 0; k0 < cut.parts; k0 += kBatch) {
            float mk[kBatch], lk[kBatch], ok[kBatch][N];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (k0 + j >= cut.parts) continue;
                const float* pk = part(k0 + j);
                mk[j] = pk[row];
                lk[j] = pk[a.part_rows + row];
                load(pk, d0, ok[j], N);
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (k0 + j < cut.parts) join_part(m, l, o, mk[j], lk[j], ok[j]);
        }
        const float inv = 1.f / l;
#pragma unroll
        for (int e = 0; e < N; e += 8)
            *reinterpret_cast<uint4*>(out + d0 + e) =
                make_uint4(pack_bf16(o[e] * inv, o[e + 1] * inv), pack_bf16(o[e + 2] * inv, o[e + 3] * inv),
                           pack_bf16(o[e + 4] * inv, o[e + 5] * inv), pack_bf16(o[e + 6] * inv, o[e + 7] * inv));
        return;
    }
    const int share = cut.parts >= 8 ? 8 : 4, mine = warp % share;
    const int span = kJoinDims * (kJoinWarps / share);  // dimensions at once
    for (int base = blockIdx.z * span; base < D; base += gridDim.z * span) {
        const int d0 = base + warp / share * kJoinDims;
        float m = -INFINITY, l = 0.f, o[kJoinDims] = {};
        if (live && d0 < D) {
            for (int k = mine; k < cut.parts; k += share) {
                const float* pk = part(k);
                float ok[kJoinDims];
                load(pk, d0, ok, kJoinDims);
                join_part(m, l, o, pk[row], pk[a.part_rows + row], ok);
            }
        }
        red[warp][0][lane] = m;
        red[warp][1][lane] = l;
#pragma unroll
        for (int e = 0; e < kJoinDims; ++e) red[warp][2 + e][lane] = o[e];
        __syncthreads();
        // each of the warps that shared dimensions writes some of them
        const int w0 = warp - mine;
        float f[kJoinWarps], top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w)
            if (w < share) top = fmaxf(top, red[w0 + w][0][lane]);
        if (top == -INFINITY) top = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            f[w] = w < share ? ex2(red[w0 + w][0][lane] - top) : 0.f;
            if (w < share) sum += f[w] * red[w0 + w][1][lane];
        }
        const float inv = 1.f / sum;
        const int per = kJoinDims / share;  // 4 or 2
        if (live && d0 < D) {
            uint32_t h[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (2 * q >= per) break;
                float x = 0.f, y = 0.f;
#pragma unroll
                for (int w = 0; w < kJoinWarps; ++w) {
                    if (f[w] == 0.f) continue;
                    x += f[w] * red[w0 + w][2 + mine * per + 2 * q][lane];
                    y += f[w] * red[w0 + w][3 + mine * per + 2 * q][lane];
                }
                h[q] = pack_bf16(x * inv, y * inv);
            }
            __nv_bfloat16* to = out + d0 + mine * per;
            if (per == 4) *reinterpret_cast<uint2*>(to) = make_uint2(h[0], h[1]);
            else *reinterpret_cast<uint32_t*>(to) = h[0];
        }
        __syncthreads();
    }
}
static_assert(kJoinDims == 2 * kJoinWarps, "two dimensions per thread at least");

bool encode_tiles(CUtensorMap* m, const void* ptr, uint64_t D, uint64_t heads, uint64_t rows, uint64_t outer,
                  uint32_t box_heads, uint32_t box_rows) {
    EncodeTiledFn fn = get_encode_fn();
    if (!fn) return false;
    const cuuint64_t gd[4] = {D, heads, rows, outer};
    const cuuint64_t gs[3] = {D * 2, heads * D * 2, rows * heads * D * 2};
    const cuuint32_t bx[4] = {64, box_heads, box_rows, 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), gd, gs, bx, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// pages of whole 8-row groups: see kGroupRows
bool encode_groups(CUtensorMap* m, const void* ptr, uint64_t D, const ChunkArgs& a) {
    EncodeTiledFn fn = get_encode_fn();
    if (!fn) return false;
    const uint64_t row = (uint64_t)a.Hkv * D * 2;
    const cuuint64_t gd[4] = {64, kGroupRows, a.Hkv * D / 64, (uint64_t)a.num_pages * a.P / kGroupRows};
    const cuuint64_t gs[3] = {row, 128, kGroupRows * row};
    const cuuint32_t bx[4] = {64, kGroupRows, (uint32_t)D / 64, (uint32_t)a.box / kGroupRows};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), gd, gs, bx, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_chunk_d(const ChunkArgs& a, const uint16_t* q, cudaStream_t st) {
    static unsigned long long configured = 0;  // bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!(configured >> dev & 1ull)) {
        // the register split assumes the launch allocation; a build that
        // allots fewer registers would leave the increase waiting forever
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, chunk_kernel<D>);
        if (e != cudaSuccess) return e;
        if (fa.numRegs < kLaunchRegs) {
            set_error_detail("chunk attention: registers at launch below the warpgroup split");
            return cudaErrorInvalidConfiguration;
        }
        e = cudaFuncSetAttribute(chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)ChunkShape<D>::kSmem());
        if (e != cudaSuccess) return e;
        configured |= 1ull << dev;
    }
    CUtensorMap tq, tqs, tk, tv, tkn, tvn;
    if (!encode_tiles(&tq, q, D, a.Hq, a.T, 1, a.grp, a.tpq) ||
        !encode_tiles(&tqs, q, D, a.Hq, a.T, 1, a.grp, a.tps > 0 ? a.tps : a.tpq) ||
        !(a.grouped ? encode_groups(&tk, a.k_pool, D, a) : encode_tiles(&tk, a.k_pool, D, a.Hkv, a.P, a.num_pages, 1, a.box)) ||
        !(a.grouped ? encode_groups(&tv, a.v_pool, D, a) : encode_tiles(&tv, a.v_pool, D, a.Hkv, a.P, a.num_pages, 1, a.box)) ||
        !encode_tiles(&tkn, a.k_new, D, a.Hkv, a.T, 1, 1, kKeys) ||
        !encode_tiles(&tvn, a.v_new, D, a.Hkv, a.T, 1, 1, kKeys)) {
        set_error_detail("chunk attention: tensor map");
        return cudaErrorInvalidValue;
    }
    const int grid = persistent_grid();
    // its launch, barriers and TMEM go under the end of the kernel before it (18.5 to
    // 16.6 us a call for one token behind 1000, call after call)
    e = launch_kernel(true, chunk_kernel<D>, dim3(grid), dim3(kChunkThreads), ChunkShape<D>::kSmem(), st, tq, tqs, tk,
                      tv, tkn, tvn, a);
    if (e != cudaSuccess) return e;
    // about 8 blocks per CTA of the cut, whatever the rows
    const int groups = a.part_rows / 32, slices = groups >= 8 ? 1 : groups >= 4 ? 4 : D / kJoinDims;
    return launch_kernel(true, chunk_join_kernel<D>, dim3(grid, groups, slices), dim3(32 * kJoinWarps), 0, st, a);
}

}  // namespace

cudaError_t launch_chunk_attention(const isd_dims* d, int T, const uint16_t* q, const uint16_t* k_new,
                                   const uint16_t* v_new, uint16_t* k_pool, uint16_t* v_pool,
                                   const int32_t* page_table, const int32_t* kv_len,
                                   const int32_t* q_start, uint16_t* out, void* ws, int32_t* err_flag,
                                   cudaStream_t st) {
    ChunkArgs a;
    a.B = d->B;
    a.T = T;
    a.Hq = d->Hq;
    a.Hkv = d->Hkv;
    a.grp = d->Hq / d->Hkv;
    a.tpq = kTileRows / a.grp;
    a.tps = 32 / a.grp;
    a.P = d->page_size;
    a.box = kKeys;  // the largest power of two up to a tile that divides the page
    while (d->page_size % a.box) a.box >>= 1;
    a.grouped = a.box >= kGroupRows;
    a.num_pages = d->num_pages;
    a.max_pages = d->max_pages_per_req;
    a.two = T > a.tpq;
    a.part_rows = chunk_part_rows(d, T);
    a.scale_log2 = d->sm_scale * 1.4426950408889634f;
    a.page_table = page_table;
    a.kv_len = kv_len;
    a.q_start = q_start;
    a.k_new = reinterpret_cast<const __nv_bfloat16*>(k_new);
    a.v_new = reinterpret_cast<const __nv_bfloat16*>(v_new);
    a.k_pool = reinterpret_cast<__nv_bfloat16*>(k_pool);
    a.v_pool = reinterpret_cast<__nv_bfloat16*>(v_pool);
    a.out = reinterpret_cast<__nv_bfloat16*>(out);
    a.cuts = static_cast<ChunkCut*>(ws);
    static_assert(sizeof(ChunkCut) == kChunkCutBytes, "workspace layout");
    a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + align_up((size_t)kMaxSMs * kChunkCutBytes, 256));
    a.err_flag = err_flag;
    return d->D == 64 ? launch_chunk_d<64>(a, q, st) : launch_chunk_d<128>(a, q, st);
}

}  // namespace isd
