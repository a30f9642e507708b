// The cut of a chunk-attention call into one range per CTA (chunk.cu): the
// requests' key tiles, flattened, on an axis of measured costs.  Plain
// arithmetic on the lengths, for the kernel and the host alike.  Sums over the
// items of a request, and with them a CTA's range, are 64-bit: the tiles grow
// with the square of its new tokens (2^31 at 1 to 12 million, by the heads of a
// group).
#pragma once

#ifdef __CUDACC__
#define ISD_CUT __host__ __device__ __forceinline__
#else
#define ISD_CUT inline
#endif

namespace isd {

constexpr int kKeys = 128;                 // keys per tile
constexpr long long kMaxKeys = 1ll << 30;  // of a request: positions and tiles fit in 32 bits
// New tokens that are put into the free rows of the last cached tile instead
// of a tile of their own.
constexpr int kMergeTokens = 16;
// Cost of a key tile and of an item's start and end on the partition axis: an
// item of two row tiles, and one of one.  Measured per CTA: 3.0 to 3.3 thousand
// cycles for a tile of two and 9.5 thousand for its ends; 1.6 thousand and 7
// thousand for one (2.5 thousand a tile when all CTAs wait for memory).
constexpr int kCost2 = 4, kEnds2 = 13, kCost1 = 2, kEnds1 = 7;

struct CutShape {
    int P, max_pages;
    int tpq;  // tokens of a tile of 128 rows
    int two;  // whether T has items of two tiles
};

// New tokens of a request if its page list can hold them, else 0 (negative
// or over-capacity length).  q_start is known to ascend within [0, T].
ISD_CUT int chunk_tokens(const CutShape& a, int kv, int n) {
    if (kv < 0) return 0;
    const long long t = (long long)kv + n;
    return t > (long long)a.max_pages * a.P || t > kMaxKeys ? 0 : n;
}

// A request as the partition sees it.
struct Request {
    int n, kv, start;
    int kvt;      // tiles with cached keys
    bool merged;  // the new tokens lie in the last of them
    int items;    // per KV head
};

ISD_CUT Request request_of(const CutShape& a, int start, int end, int kv) {
    Request r;
    r.start = start;
    r.kv = kv;
    r.n = chunk_tokens(a, kv, end - start);
    r.kvt = ((kv > 0 ? kv : 0) + kKeys - 1) / kKeys;
    r.merged = r.n <= kMergeTokens && r.n <= r.kvt * kKeys - kv;
    r.items = (r.n + 2 * a.tpq - 1) / (2 * a.tpq);
    return r;
}

struct Item {
    int i0, i1;  // its tokens
    bool two;
    int nt, w, cost;  // key tiles, cost of one, of all
};

// Cost of a request's items of one KV head.
ISD_CUT long long head_cost(const CutShape& a, const Request& r) {
    if (r.items == 0) return 0;
    // all items but the last have two tiles; their new keys' tiles one by one
    const int span = 2 * a.tpq, full = r.items - 1;
    long long fresh = 0;
    if (!r.merged)
        for (int q = 0, end = span; q < full; ++q, end += span) fresh += (end + kKeys - 1) / kKeys;
    long long c = (long long)full * (kCost2 * (long long)r.kvt + kEnds2) + kCost2 * fresh;
    const bool two = r.n - full * span > a.tpq;
    const int nt = r.kvt + (r.merged ? 0 : (r.n + kKeys - 1) / kKeys);
    return c + (two ? kCost2 * nt + kEnds2 : kCost1 * nt + kEnds1);
}

ISD_CUT Item item_of(const CutShape& a, const Request& r, int q) {
    Item it;
    it.i0 = q * 2 * a.tpq;
    it.i1 = r.n < it.i0 + 2 * a.tpq ? r.n : it.i0 + 2 * a.tpq;
    it.two = it.i1 - it.i0 > a.tpq;
    it.nt = r.kvt + (r.merged ? 0 : (it.i1 + kKeys - 1) / kKeys);
    it.w = it.two ? kCost2 : kCost1;
    it.cost = it.w * it.nt + (it.two ? kEnds2 : kEnds1);
    return it;
}

// CTAs of `grid` that get a range, and the start of one's: every CTA between
// the ends of a cut item has a tile of it.
ISD_CUT int cut_ctas(const CutShape& a, long long total, int grid) {
    const long long most = a.two ? total / kCost2 : total / kCost1;
    return most < 1 ? 1 : most < grid ? (int)most : grid;
}
ISD_CUT long long cut_start(long long total, int ctas, int cta) {
    if (total < (1 << 23)) return (unsigned)total * (unsigned)cta / (unsigned)ctas;  // fits in 32 bits
    return total * cta / ctas;
}
// The CTA whose range holds position x.
ISD_CUT int cut_owner(long long total, int ctas, long long x) { return (int)(((x + 1) * ctas - 1) / total); }

// The item (of KV head g, number q) of a request that holds the position `rem`
// past the request's start; returns what of `rem` is left past the item's.
ISD_CUT int cut_item(const CutShape& a, const Request& r, long long head, long long rem, int& g, int& q) {
    for (g = 0; rem >= head; ++g) rem -= head;
    q = 0;
    for (int w; (w = item_of(a, r, q).cost) <= rem; ++q) rem -= w;
    return (int)rem;
}

// The tiles [t0, t1) of an item that starts at `start` in a range of length
// `len` (none: only a part of its ends lies there).
ISD_CUT void cut_tiles(const Item& it, long long start, long long len, int& t0, int& t1) {
    // (divisions by constants: the walk is on the path to a CTA's first load)
    const auto ceil_of = [&](long long x) { return it.two ? (x + kCost2 - 1) / kCost2 : (x + kCost1 - 1) / kCost1; };
    t0 = start < 0 ? (int)ceil_of(-start) : 0;
    const long long end = ceil_of(len - start);
    t1 = it.nt < end ? it.nt : (int)end;
}

}  // namespace isd
