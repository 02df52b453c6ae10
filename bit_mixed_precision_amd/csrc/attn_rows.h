// Which rows of q a sequence's queries are, from device values that may be
// anything: plain integers, so that the host can check it too.
#pragma once

#ifdef __HIPCC__
#define BQ_HOST_DEVICE __host__ __device__ inline
#else
#define BQ_HOST_DEVICE inline
#endif

namespace bq {

struct QueryRows {
    int first;  // row of q of the sequence's first query
    int len;    // its queries: query i stands at key seq_len - len + i
    int count;  // those that are computed, the first ones
};

// Queries [start, end) taken within [0, total], the first `most` of them
// computed.  Both ends are brought into the range before they are subtracted:
// the difference of two arbitrary values would pass 32 bits.
// first + count <= first + len <= total.
BQ_HOST_DEVICE QueryRows query_rows_of(int start, int end, int total, int most)
{
    const int first = start < 0 ? 0 : start < total ? start : total;
    const int stop = end < first ? first : end < total ? end : total;
    const int len = stop - first;
    return {first, len, len < most ? len : most};
}

}  // namespace bq
