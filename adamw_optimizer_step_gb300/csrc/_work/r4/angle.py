# host arithmetic of rope_run's turns, against rationals with a 60-digit pi
import math
from fractions import Fraction
PI=Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
def turns_now(f):
    turn=f/6.283185307179586476925286766559
    fr=turn-math.floor(turn)
    return 0 if fr>=1.0 else int(math.ldexp(fr,64))
def turns_new(f):
    turn=abs(f)/6.283185307179586476925286766559
    fr=turn-math.floor(turn)
    v=int(math.ldexp(fr,64))
    return v if f>=0 else (-v)%2**64
def err(turns,t,f):
    got=Fraction((t*turns)%2**64,2**64); want=Fraction(t)*Fraction(f)/(2*PI)
    d=got-want; d-=round(d)
    return abs(float(d*2*PI))
for fn in (turns_now,turns_new):
    print(fn.__name__)
    for f in (1.0,0.3,1e-3,2.0**-10,1e-4,-1.0,-0.3,-1e-4,-1e-8, 1e-8,1000.3,-1000.3):
        row=[]
        for t in (2**24+1,2**31+3,2**35+9,2**40+12345,-(2**33)-7):
            e=err(fn(f),t,f); b=abs(t)*(abs(f)*2.0**-52+2.0**-61)
            row.append("%.1e(%.2f)"%(e,e/b))
        print("%9g"%f,*row)
