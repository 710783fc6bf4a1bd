// es_segments.h -- which chunks of a row a segment of linear attention takes,
// and which segment's state enters it.  Plain C++, for the kernels and for the
// host alike (tests/test_attention_segments.py walks every case on the CPU).
#pragma once

#ifdef __CUDACC__
#define ES_SEGMENTS_HD __host__ __device__ __forceinline__
#else
#define ES_SEGMENTS_HD inline
#endif

namespace es {

// A call cuts every row into the same n_segs segments of seg_chunks chunks; a
// row shorter than the longest has nothing in the segments past its last one.
struct SegmentPart {
    int c0, c1;                  // its chunks [c0, c1) of the row's, c0 >= c1: none
    int last;                    // the row's last segment with chunks (0 for a row without any)
    bool begins, ends;           // the run starts in it, ends in it
    int entry;                   // place of the state entering it among the row's n_segs kept states; -1: none
};

// The place of a segment's successor's state is its own.  The run's last
// segment has no successor: its place holds the run's first state.  A segment
// past the row's last takes no state: its predecessor along a reversed run need
// not exist, nor the place of its state.
ES_SEGMENTS_HD SegmentPart segment_part(int seg, int n_segs, int seg_chunks, int chunks, bool reverse) {
    SegmentPart p;
    p.c0 = seg * seg_chunks;
    p.c1 = chunks < p.c0 + seg_chunks ? chunks : p.c0 + seg_chunks;
    p.last = chunks > 0 ? (chunks - 1) / seg_chunks : 0;
    p.begins = reverse ? seg == p.last : seg == 0;
    p.ends = reverse ? seg == 0 : seg == p.last;
    if (n_segs == 1 || seg > p.last) p.entry = -1;
    else if (p.begins) p.entry = reverse ? 0 : p.last;
    else p.entry = reverse ? seg + 1 : seg - 1;
    return p;
}

}  // namespace es
