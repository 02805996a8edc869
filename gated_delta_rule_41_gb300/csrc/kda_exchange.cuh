// The turns of an exchange among the K CTAs of a cluster: in each, every CTA sends one message to all
// (itself too) and waits for all K messages, which count on a barrier of its own shared memory, one
// barrier for the even turns and one for the odd.  Turns 0 and 1 are expected from the start, turn t + 2
// once those of turn t are here.  A message of turn t + 2 is sent by a CTA that has all of turn t + 1, so
// by then its receiver has read those of turn t and expects it.
//
// A wait may give up.  Its CTA is then lost: it waits and expects no more, but sends as before (in the
// scans' loops a condition around the sends takes 4 us of 81).  So each CTA is sent a message of every
// turn by each, and its end can wait for all of them: nothing may be on its way to a CTA that has ended.
// Messages of a lost CTA that come too early are taken for others of their barrier; the results are not to
// be used.  A barrier counts fewer than 2^20 bytes: with 512 a message, that holds for any order of messages
// where K times the turns are at most 4064 (2^19 tokens of a scan).  Where more than a barrier counts may be
// on its way to a lost CTA, that lets its waits' limit pass instead.
//
// (Without a GPU the tests run this on threads.)
#pragma once

#ifdef __CUDACC__
#define KDA_EXCHANGE_FN __device__ __forceinline__
#else
#define KDA_EXCHANGE_FN inline
#endif

namespace kda {

// The end of a CTA that was lost in turn `lost`, once all CTAs have sent their messages of all turns (a
// barrier of the cluster says so).  It has expected those of turns up to lost + 1.  The others are now
// expected too, in whatever phase each barrier is: that of the last expected turn, which then ends when
// all is here, or the next, which ends then and with an arrival more.  (A CTA that is not lost has had all
// that is sent to it.)
// Port, of one CTA:
//   wait(turn)            for the end of this turn's phase; false if it gives up again
//   expect(turn, n)       n more messages of each CTA on this turn's barrier, whatever its phase
//   arrive(turn)          the arrival that a phase of this turn's barrier needs, and none before
//   pause()               for as long as a wait's limit
template <typename Port>
KDA_EXCHANGE_FN void exchange_drain(Port& port, int K, int turns, int lost) {
    constexpr int kMost = (1 << 20) / 512 - 16;   // messages, beside those of a turn
    if ((long long)(turns - 1 - lost) / 2 * K > kMost) {
        port.pause();
        return;
    }
    for (int turn = lost; turn <= lost + 1 && turn < turns; ++turn) {
        port.expect(turn, (turns - 1 - turn) / 2);
        if (!port.wait(turn)) continue;
        port.arrive(turn);
        port.wait(turn + 2);
    }
}

}  // namespace kda
